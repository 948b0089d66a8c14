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

// The power of two that brings m into [2^TO, 2^(TO + 1)), at most 2^100; and the
// exact inverse of such a power.
template <int TO>
__device__ __forceinline__ float pow2_to(float m) {
    const int e = static_cast<int>(__float_as_uint(m) >> 23) & 255;
    const int f = 254 + TO - e;
    return __uint_as_float(static_cast<uint32_t>(f < 227 ? f : 227) << 23);
}
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// What prep leaves for one (sequence, group, chunk), in fragments of 64 lanes x
// 8 fp16 (1 KB): C (rows: tokens, k: entries), B transposed (rows: entries, k:
// tokens) and G (rows: tokens, k: tokens; the six k-steps at or below the
// diagonal), each as hi and, where wanted, lo; then 2^-s per token of B and C.
template <int N, bool FINE>
struct Shared {
    static constexpr int CF = 2 * (N / 16), BF = 4 * (N / 32), GF = 6;   // fragments of one part
    static constexpr int kC = 0, kCl = CF, kB = FINE ? 2 * CF : CF, kBl = kB + BF, kG = kBl + BF, kGl = kG + GF;
    static constexpr int kFrags = kG + (FINE ? 2 : 1) * GF;
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
            const float s = pow2_to<2>(m);
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

struct ChunkArgs {
    SsmArgs p;
    const int32_t* lengths;
    const _Float16* shared;   // prep's output
    float* seg_state;         // [B][H][segments][P][N]
    float* seg_decay;         // [B][H][segments] log2 of the segment's decay
    int T, B, H, G, P, C, nc, segs, chunks_per_seg;
};

// OUT: form the outputs.  EXACT: the state's products in two fp16 parts.  With
// segments, OUT without EXACT serves bf16 outputs (the state comes from join).
template <int N, typename Act, bool FINE, bool OUT, bool EXACT>
__global__ __launch_bounds__(256) void ssm_chunk_kernel(ChunkArgs a) {
    using Sh = Shared<N, FINE>;
    using Qd = Quad<Act>;
    constexpr int NT = N / 32;
    __shared__ __align__(16) float factors[4][6][Q];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int hi = lane >> 5, c = lane & 31;
    const int slices = a.P / 32;
    int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + wave;
    const int slice = static_cast<int>(id % slices);
    id /= slices;
    const int h = static_cast<int>(id % a.H);
    id /= a.H;
    const int seg = static_cast<int>(id % a.segs);
    const int seq = static_cast<int>(id / a.segs);
    if (seq >= a.B)
        return;
    const int len = a.lengths ? a.lengths[seq] : a.T;
    if (len < 1 || len > a.T)
        return;
    const int last = (len + Q - 1) / Q;
    const int ch0 = seg * a.chunks_per_seg;
    const int ch1 = ch0 + a.chunks_per_seg < last ? ch0 + a.chunks_per_seg : last;
    if (ch0 >= ch1)
        return;
    const bool split = a.segs > 1;

    const int g = h / (a.H / a.G);
    const int chan = h * a.P + slice * 32 + c;   // this lane's state row, as an x channel
    const Act* xs = static_cast<const Act*>(a.p.x) + static_cast<size_t>(seq) * a.T * a.C + chan;
    const Act* tail = static_cast<const Act*>(a.p.tail_in) + (static_cast<size_t>(seq) * a.C + chan) * 4;
    const float* dts = a.p.dt + static_cast<size_t>(seq) * a.T * a.H + h;
    float wf[4];
    Qd::to_float(Qd::load(static_cast<const Act*>(a.p.w) + static_cast<size_t>(chan) * 4), wf);
    const float bf = a.p.bias ? widen(static_cast<const Act*>(a.p.bias)[chan]) : 0.0f;
    const float dtb = a.p.dt_bias ? a.p.dt_bias[h] : 0.0f;
    const double rate = static_cast<double>(rate2(a.p.A[h]));
    const float skip = a.p.D ? a.p.D[h] : 0.0f;
    const size_t yrow = static_cast<size_t>(a.H) * a.P;
    const size_t ybase = static_cast<size_t>(seq) * a.T * yrow + chan;

    float* fF = factors[wave][0];   // d * 2^-s_B
    float* fW = factors[wave][1];   // 2^(c_last - c)
    float* fE = factors[wave][2];   // 2^c
    float* fS = factors[wave][3];   // 2^-s_C
    float* fH = factors[wave][4];   // c, high and low part
    float* fL = factors[wave][5];

    // the state, transposed: S[nt][v] is entry 32 nt + 8 (v / 4) + 4 hi + v % 4 of this lane's row, times `unit`
    f16v S[NT];
    float unit = 1.0f;
    const size_t head = static_cast<size_t>(seq) * a.H + h;
    const size_t row_off = static_cast<size_t>(slice * 32 + c) * N + 4 * hi;
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

    double seg_sum = 0.0;
    for (int ch = ch0; ch < ch1; ++ch) {
        const int t0 = ch * Q;
        const _Float16* sh = a.shared + ((static_cast<size_t>(seq) * a.G + g) * a.nc + ch) * Sh::kHalfs;
        const float* scales = reinterpret_cast<const float*>(sh + Sh::kFrags * 512);
        // x, with the three tokens before each run of four
        float xr[8][7];
        if (t0 > 0 && t0 + Q <= len) {
            const Act* p = xs + static_cast<size_t>(t0 + 4 * hi) * a.C;
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    xr[r][e] = widen(p[static_cast<int64_t>(8 * r + e - 3) * a.C]);
        } else {
            float tw[4];
            Qd::to_float(Qd::load(tail), tw);
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int e = 0; e < 7; ++e) {
                    const int t = t0 + 8 * r + 4 * hi + e - 3;
                    const float v = widen(xs[static_cast<size_t>(t < 0 ? 0 : t < len ? t : len - 1) * a.C]);
                    xr[r][e] = t >= 0 ? (t < len ? v : 0.0f) : t == -1 ? tw[3] : t == -2 ? tw[2] : tw[1];
                }
        }
        // the chunk's step sizes and decays, one token per lane
        double total;
        {
            const int t = t0 + lane;
            const float d = t < len ? step_size(dts[static_cast<size_t>(t) * a.H] + dtb) : 0.0f;
            const double cum = wave_scan(static_cast<double>(d) * rate, lane);
            total = __shfl(cum, 63);
            fF[lane] = d * scales[lane];
            fW[lane] = __builtin_amdgcn_exp2f(static_cast<float>(total - cum));
            if (OUT) {
                const float ch_ = static_cast<float>(cum);
                fE[lane] = __builtin_amdgcn_exp2f(ch_);
                fS[lane] = scales[Q + lane];
                fH[lane] = ch_;
                fL[lane] = static_cast<float>(cum - static_cast<double>(ch_));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        const float decay = __builtin_amdgcn_exp2f(static_cast<float>(total));
        seg_sum += total;

        // conv; X' and the largest of it and of X'' in this row
        float xc[32], xp[32];
        float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float4 F = *reinterpret_cast<const float4*>(fF + 8 * r + 4 * hi);
            const float4 W = *reinterpret_cast<const float4*>(fW + 8 * r + 4 * hi);
            const float ff[4] = {F.x, F.y, F.z, F.w}, ww[4] = {W.x, W.y, W.z, W.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float win[4] = {xr[r][i], xr[r][i + 1], xr[r][i + 2], xr[r][i + 3]};
                const float v = conv_bias_silu(wf, win, bf);
                xc[4 * r + i] = v;
                xp[4 * r + i] = v * ff[i];
                m1 = fmaxf(m1, fabsf(xp[4 * r + i]));
                m2 = fmaxf(m2, fabsf(xp[4 * r + i] * ww[i]));
            }
        }
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
        const float room = fminf(pow2_to<60>(ms * inverse_pow2(unit)), unit * 0x1p60f);

        if (OUT) {
            const float sx = fminf(pow2_to<8>(m1), room);
            const float ss = pow2_to<8>(ms);   // on top of `unit`
            f16v Y[2] = {zero16(), zero16()};
            // C S0^T
#pragma unroll
            for (int ks = 0; ks < N / 16; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = S[ks / 2][8 * (ks % 2) + e] * ss;
                h8 bh, bl;
                parts8<FINE>(v, bh, bl);
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const h8 ah = ld_frag(sh, Sh::kC + it * (N / 16) + ks, lane);
                    Y[it] = mma(ah, bh, Y[it]);
                    if (FINE) {
                        Y[it] = mma(ah, bl, Y[it]);
                        Y[it] = mma(ld_frag(sh, Sh::kCl + it * (N / 16) + ks, lane), bh, Y[it]);
                    }
                }
            }
            const float ratio = sx * inverse_pow2(ss) * inverse_pow2(unit);
#pragma unroll
            for (int it = 0; it < 2; ++it)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 E = *reinterpret_cast<const float4*>(fE + 32 * it + 8 * q + 4 * hi);
                    Y[it][4 * q] *= E.x * ratio;
                    Y[it][4 * q + 1] *= E.y * ratio;
                    Y[it][4 * q + 2] *= E.z * ratio;
                    Y[it][4 * q + 3] *= E.w * ratio;
                }
            // (M . G) X'
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                float v[8], cj[8], lj[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = xp[8 * ks + e] * sx;
                    cj[e] = fH[16 * ks + kperm(hi, e)];
                    if (FINE)
                        lj[e] = fL[16 * ks + kperm(hi, e)];
                }
                h8 bh, bl;
                parts8<FINE>(v, bh, bl);
#pragma unroll
                for (int it = ks / 2; it < 2; ++it) {
                    const float ci = fH[32 * it + c];
                    const float li = FINE ? fL[32 * it + c] : 0.0f;
                    const h8 gh = ld_frag(sh, Sh::kG + Sh::g_frag(it, ks), lane);
                    h8 gl = gh;
                    if (FINE)
                        gl = ld_frag(sh, Sh::kGl + Sh::g_frag(it, ks), lane);
                    float m[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float arg = ci - cj[e];
                        float gv = static_cast<float>(gh[e]);
                        if (FINE) {
                            arg += li - lj[e];
                            gv += static_cast<float>(gl[e]);
                        }
                        m[e] = gv * __builtin_amdgcn_exp2f(arg);
                        if (it == ks / 2)   // a block on the diagonal
                            m[e] = 16 * ks + kperm(hi, e) <= 32 * it + c ? m[e] : 0.0f;
                    }
                    h8 mh, ml;
                    parts8<FINE>(m, mh, ml);
                    Y[it] = mma(mh, bh, Y[it]);
                    if (FINE) {
                        Y[it] = mma(mh, bl, Y[it]);
                        Y[it] = mma(ml, bh, Y[it]);
                    }
                }
            }
            const float back = inverse_pow2(sx);
            Act* yp = static_cast<Act*>(a.p.y) + ybase;
            const Act* zp = static_cast<const Act*>(a.p.z) + (a.p.z ? ybase : 0);
#pragma unroll
            for (int it = 0; it < 2; ++it)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int tr = 32 * it + 8 * q + 4 * hi;
                    const float4 Sc = *reinterpret_cast<const float4*>(fS + tr);
                    const float sc[4] = {Sc.x, Sc.y, Sc.z, Sc.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = t0 + tr + i;
                        if (t < len) {
                            float o = __builtin_fmaf(skip, xc[16 * it + 4 * q + i], Y[it][4 * q + i] * (sc[i] * back));
                            if (a.p.z)
                                o *= silu(widen(zp[static_cast<size_t>(t) * yrow]));
                            narrow(o, yp[static_cast<size_t>(t) * yrow]);
                        }
                    }
                }
        }

        if (!OUT || !split || ch + 1 < ch1) {
            // S1: the row's unit becomes that of X'' unless the state is too large for it
            const float s2 = fminf(pow2_to<8>(m2), room);
            const float keep = decay * (s2 * inverse_pow2(unit));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    S[nt][v] *= keep;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = xp[8 * ks + e] * (fW[16 * ks + kperm(hi, e)] * s2);
                h8 bh, bl;
                parts8<EXACT>(v, bh, bl);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const h8 ah = ld_frag(sh, Sh::kB + nt * 4 + ks, lane);
                    S[nt] = mma(ah, bh, S[nt]);
                    if (EXACT) {
                        S[nt] = mma(ah, bl, S[nt]);
                        S[nt] = mma(ld_frag(sh, Sh::kBl + nt * 4 + ks, lane), bh, S[nt]);
                    }
                }
            }
            unit = s2;
        }
        // the factors are rewritten by the next chunk
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
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
    if (split && slice == 0 && lane == 0)
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
    size_t n = up256(static_cast<size_t>(g.B) * g.G * nc * shared_halfs(g) * sizeof(_Float16));
    if (segs > 1)
        n += up256(static_cast<size_t>(g.B) * g.H * segs * g.P * g.N * 4) + up256(static_cast<size_t>(g.B) * g.H * segs * 4);
    return n;
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
    const ChunkArgs a{p, lengths, shared, seg_state, seg_decay, T, g.B, g.H, g.G, g.P, g.C, nc, segs, per};
    const int64_t waves = static_cast<int64_t>(g.B) * g.H * (g.P / 32) * segs;
    const dim3 grid(static_cast<unsigned>((waves + 3) / 4)), block(256);
    if (segs == 1) {
        hipLaunchKernelGGL((ssm_chunk_kernel<N, Act, FINE, true, true>), grid, block, 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((ssm_chunk_kernel<N, Act, FINE, false, true>), grid, block, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    const int quads = g.P * N / 4;
    const int64_t threads = static_cast<int64_t>(g.B) * g.H * quads;
    hipLaunchKernelGGL(ssm_join_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), block, 0, s, a, quads);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    hipLaunchKernelGGL((ssm_chunk_kernel<N, Act, FINE, true, FINE>), grid, block, 0, s, a);
    return hipGetLastError();
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
