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
//          group's B and C channels, and G, once for all heads of the group;
//          beside them the step sizes d and the sums c, per head.
//   chunk  one wave per (sequence, head, 32 rows of the state, segment of
//          chunks): the state stays transposed in accumulators (entries down,
//          rows across) from chunk to chunk, and since a lane's accumulators
//          of one product are its operand of the next (the fragment order
//          below), no value passes between lanes.
//   A prompt is cut into segments where there are too few (sequence, head)
//   pairs to fill the chip: `state` forms each segment's own state from zero
//   and leaves the convolved x behind, `join` adds the states up (the decay of
//   a head is one number, so they combine by a scaled sum), and the output pass
//   runs from the states that enter the segments.
//
// Precision.  fp16 matrix products with fp32 accumulation.  Every operand is
// scaled by a power of two that keeps its largest value in range: B and C per
// token, X' and X'' per state row and chunk, the state per row; scaling is
// exact and undone on the accumulators.  Products that reach the state or fp32
// outputs take each operand as the sum of two fp16 numbers (22 bits) and three
// matrix products, so that the state is as exact as one kept in fp32.  Outputs
// that are rounded to bf16 take one fp16 number (11 bits against bf16's 8).  Each
// of X', X'' and the state has its own scale, from its own largest value: a step
// that wipes the state leaves X'' far below X', and the state far below both.
// Within a chunk M . G has none: an output whose terms M takes below 2^-14 keeps
// fewer bits, 2^-24 (bf16, with the steps of the segments' pass in fp16, 2^-16) of
// the chunk's largest products being what is left out at most.
#include <algorithm>
#include <type_traits>

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
// A uniform base and a lane's 32-bit byte offset: one register of addresses
// instead of two.
template <typename T>
__device__ __forceinline__ T& at(const void* base, uint32_t bytes) {
    return *reinterpret_cast<T*>(const_cast<char*>(static_cast<const char*>(base)) + bytes);
}
__device__ __forceinline__ h8 ld_frag(const _Float16* m, int frag, int lane) {
    return at<const h8>(m + frag * 512, static_cast<uint32_t>(lane) * 16u);
}
__device__ __forceinline__ void st_frag(_Float16* m, int frag, int lane, h8 v) {
    at<h8>(m + frag * 512, static_cast<uint32_t>(lane) * 16u) = v;
}
// v = hi + lo in fp16 (21 bits and more where v is well inside fp16's range): hi
// is v cut to fp16, two at a time by one instruction, and lo the rest, formed by
// the mixed multiply-add that reads an fp16 operand as it is (the factor -1 is
// hidden, or the compiler makes a conversion and a subtraction of it).  Rounding
// hi instead would not do with an ordinary conversion: the compiler may fuse the
// product that v comes from into it, and hi is now and then not what lo is the
// rest of.
__device__ __forceinline__ void split8(const float (&v)[8], h8& hi, h8& lo) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    float minus = -1.0f;
    asm("" : "+s"(minus));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const h2 h = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_pkrtz(v[e], v[e + 1]));
        hi[e] = h.x;
        hi[e + 1] = h.y;
        lo[e] = static_cast<_Float16>(__builtin_fmaf(static_cast<float>(h.x), minus, v[e]));
        lo[e + 1] = static_cast<_Float16>(__builtin_fmaf(static_cast<float>(h.y), minus, v[e + 1]));
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
// Caps of the scales.  A row of B, C, x or X' whose largest value is below 2^-38,
// or of X'' below 2^-56, loses relative precision to fp16's absolute 2^-24 at that
// scale; in return no product of scales and states leaves fp32's range.
constexpr int kMostBC = 40, kMostX = 24, kMostF = 24, kMostW = 64, kMostS = 100;
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }
// The unit of a row whose largest value is m, where values of at most `carried` in
// the unit before are to be brought to it: they end below 2^100, and the ratio of the
// units is finite.
__device__ __forceinline__ float unit_for(float m, float unit, float carried) {
    const float most = unit * 0x1p60f * __builtin_amdgcn_rcpf(carried) * 0x1p40f;
    const float cut = __uint_as_float(__float_as_uint(most) & 0x7F800000u);
    return fminf(fminf(pow2_to<8, kMostW>(m), unit * 0x1p120f), fmaxf(cut, 0x1p-120f));
}
// The largest that a chunk's X''^T B comes to: 64 products of less than 2^9 and 2^3.
constexpr float kMostUpdate = 0x1p18f;

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

// ------------------------------------------------------------ conv

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

// A wave's tile in LDS: 64 tokens x 32 channels of x after the four tokens
// before them; later 32 tokens of y in fp32.  The pitch (40 elements) puts the
// two lane halves' rows, four apart, into different banks.
template <typename Act>
struct Tile {
    static constexpr int kUnit = 16 / sizeof(Act);     // channels per 16 bytes
    static constexpr int kPerRow = 32 / kUnit;         // 16-byte units per row; also units per lane of 64 rows
    static constexpr int kRowStep = 64 / kPerRow;      // rows between a lane's units
    static constexpr int kPitch = 40;
    static constexpr int kRows = Q + 4;
    static constexpr int kBytes = kRows * kPitch * sizeof(Act);
    static_assert(kBytes >= 32 * kPitch * 4, "half a tile of fp32 outputs fits");
};

// One channel's taps.  bf16 keeps them in pairs for the packed dot product (fp32
// accumulation, within one rounding of the exact sum), in the two alignments
// that a window can have against pairs of tokens; the taps that a pair has no
// part in are zeros.
template <typename Act>
struct Taps;
template <>
struct Taps<uint16_t> {
    uint32_t z0, w12, w3z, w01, w23;
    float bias;
    __device__ void load(const uint16_t* w, const uint16_t* b, int ch) {
        const uint2 r = *reinterpret_cast<const uint2*>(w + static_cast<size_t>(ch) * 4);
        w01 = r.x;
        w23 = r.y;
        z0 = r.x << 16;
        w12 = (r.x >> 16) | (r.y << 16);
        w3z = r.y >> 16;
        bias = b ? widen(b[ch]) : 0.0f;
    }
};
template <>
struct Taps<float> {
    float w[4];
    float bias;
    __device__ void load(const float* p, const float* b, int ch) {
        const float4 r = *reinterpret_cast<const float4*>(p + static_cast<size_t>(ch) * 4);
        w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        bias = b ? b[ch] : 0.0f;
    }
};
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, a), __builtin_bit_cast(b2, b), c, false);
}

// SiLU(conv) of run r of this lane's channel: tokens 8 r + 4 hi .. + 3 of the tile,
// as what is read for it and each of the four.
// bf16: the transposing LDS read gives a lane four tokens of its channel; the
// lane supplies the address of four channels of one token.
template <typename Act>
struct Run;
template <>
struct Run<uint16_t> {
    uint2 a, b;
    __device__ void load(const uint16_t* tile, int r, int lane) {
        typedef __attribute__((address_space(3))) s4* lds4;
        constexpr int kPitch = Tile<uint16_t>::kPitch;
        const int row = (lane >> 5) * 4 + ((lane & 15) >> 2);
        const uint16_t* p = tile + row * kPitch + (lane & 16) + (lane & 3) * 4 + 8 * r * kPitch;
        a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p));
        b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * kPitch)));
    }
    __device__ float out(const Taps<uint16_t>& k, int i) const {
        return silu(i == 0   ? dot2(b.x, k.w3z, dot2(a.y, k.w12, dot2(a.x, k.z0, k.bias)))
                    : i == 1 ? dot2(b.x, k.w23, dot2(a.y, k.w01, k.bias))
                    : i == 2 ? dot2(b.y, k.w3z, dot2(b.x, k.w12, dot2(a.y, k.z0, k.bias)))
                             : dot2(b.y, k.w23, dot2(b.x, k.w01, k.bias)));
    }
};
template <>
struct Run<float> {
    float v[7];
    __device__ void load(const float* tile, int r, int lane) {
        const float* p = tile + ((lane >> 5) * 4 + 8 * r + 1) * Tile<float>::kPitch + (lane & 31);
#pragma unroll
        for (int e = 0; e < 7; ++e)
            v[e] = p[e * Tile<float>::kPitch];
    }
    __device__ float out(const Taps<float>& k, int i) const {
        const float win[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
        return conv_bias_silu(k.w, win, k.bias);
    }
};
template <typename Act>
__device__ __forceinline__ void conv_run(const Act* tile, const Taps<Act>& k, int r, int lane, float (&out)[4]) {
    Run<Act> run;
    run.load(tile, r, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = run.out(k, i);
}

// A wave's path of x from memory through its tile, a chunk at a time.
template <typename Act>
struct Stream {
    using Tl = Tile<Act>;
    Act* tile;
    const Act* x;     // the sequence's rows, at the wave's first channel
    int C, len, urow, ucol, lane;
    u4 unit[Tl::kPerRow];
    u4 keep;          // the tile's last four rows (lanes 0 .. 4 * kPerRow - 1)

    __device__ void load(int t0) {   // rows behind the sequence's end are the last row again
#pragma unroll
        for (int k = 0; k < Tl::kPerRow; ++k) {
            const int r = min(urow + k * Tl::kRowStep, len - 1 - t0);
            unit[k] = at<const u4>(x + static_cast<size_t>(t0) * C,
                                   static_cast<uint32_t>(r * C + ucol) * static_cast<uint32_t>(sizeof(Act)));
        }
    }
    // the four rows before t0: of the sequence, or the conv tail of these channels
    __device__ void begin(const Act* tail, int t0) {
        if (t0 > 0) {
            if (lane < 4 * Tl::kPerRow)
                keep = *reinterpret_cast<const u4*>(x + static_cast<size_t>(t0 - 4 + lane / Tl::kPerRow) * C +
                                                    lane % Tl::kPerRow * Tl::kUnit);
        } else {
            if (lane < 32) {
                const typename Quad<Act>::raw r = Quad<Act>::load(tail + lane * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tile[j * Tl::kPitch + lane] = Quad<Act>::elem(r, j);
            }
            wave_sync();
            save(0);
        }
    }
    __device__ void save(int row) {
        if (lane < 4 * Tl::kPerRow)
            keep = *reinterpret_cast<const u4*>(tile + (row + lane / Tl::kPerRow) * Tl::kPitch +
                                                lane % Tl::kPerRow * Tl::kUnit);
    }
    __device__ void store() {
        if (lane < 4 * Tl::kPerRow)
            *reinterpret_cast<u4*>(tile + lane / Tl::kPerRow * Tl::kPitch + lane % Tl::kPerRow * Tl::kUnit) = keep;
#pragma unroll
        for (int k = 0; k < Tl::kPerRow; ++k)
            *reinterpret_cast<u4*>(tile + (4 + urow + k * Tl::kRowStep) * Tl::kPitch + ucol) = unit[k];
    }
};
template <typename Act>
__device__ __forceinline__ Stream<Act> make_stream(Act* tile, const Act* x, int C, int len, int lane) {
    Stream<Act> s;
    s.tile = tile;
    s.x = x;
    s.C = C;
    s.len = len;
    s.lane = lane;
    s.urow = lane / Tile<Act>::kPerRow;
    s.ucol = lane % Tile<Act>::kPerRow * Tile<Act>::kUnit;
    s.keep = u4{0, 0, 0, 0};
    return s;
}

// ------------------------------------------------------------ prep

// What prep leaves for one (sequence, group, chunk), in fragments of 64 lanes x
// 8 fp16 (1 KB): C (rows: tokens, k: entries), G (rows: tokens, k: tokens; the
// six k-steps at or below the diagonal) and B transposed (rows: entries, k:
// tokens), each as hi and, where wanted, lo; then 2^-s per token of B and C.
template <int N, bool FINE>
struct Shared {
    static constexpr int CF = 2 * (N / 16), BF = 4 * (N / 32), GF = 6;   // fragments of one part
    static constexpr int kC = 0, kCl = CF, kG = FINE ? 2 * CF : CF, kGl = kG + GF, kB = kG + (FINE ? 2 : 1) * GF,
                         kBl = kB + BF, kFrags = kBl + BF;
    static constexpr size_t kHalfs = static_cast<size_t>(kFrags) * 512 + 256;   // scales: 128 floats
    static __device__ int g_frag(int it, int ks) { return it == 0 ? ks : 2 + ks; }
};

struct ChunkArgs {
    SsmArgs p;
    const int32_t* lengths;
    int32_t* status;
    _Float16* shared;         // per (sequence, group, chunk): Shared<>
    float* steps;             // [B][H][nc][3][64]: d, then c as a high and a low part
    float* seg_state;         // [B][H][segments][P][N]
    float* seg_decay;         // [B][H][segments] log2 of the segment's decay
    char* conv;               // [B][H][nc][P / 32] convolved x (Conv<>)
    int T, B, H, G, P, C, nc, segs, chunks_per_seg, by_xcd;
};

// Largest magnitude of a 16-lane row's values, in all its lanes.  As integers,
// magnitudes keep their order, and a step is one instruction (a float maximum
// of a moved value takes four: prep 81 -> 68 us at 16 groups).
template <int CTRL>
__device__ __forceinline__ uint32_t max_of_moved(uint32_t v) {
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t row_max_bits(float v) {
    uint32_t m = __float_as_uint(v) & 0x7FFFFFFFu;
    m = max_of_moved<0xB1>(m);
    m = max_of_moved<0x4E>(m);
    m = max_of_moved<0x141>(m);
    return max_of_moved<0x140>(m);
}
__device__ __forceinline__ float row_max(float v) { return __uint_as_float(row_max_bits(v)); }
__device__ __forceinline__ float wave_max(float v) {
    const int m = static_cast<int>(row_max_bits(v));
    uint32_t r = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        r = max(r, static_cast<uint32_t>(__builtin_amdgcn_readlane(m, 16 * k)));
    return __uint_as_float(r);
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

constexpr int kStepHeads = 16;   // heads per workgroup of the step sizes

// Step sizes and summed decays of a chunk's tokens.  c is summed in fp64: what
// matters are differences of it, also where it is large.  A token's part of it
// ends at -160, where the decay is 0 in fp32 whatever else is added, so that the
// high part alone (all that bf16 outputs use) is within 2^-11 of c.
constexpr float kLeastDecay = -160.0f;
__device__ void steps_part(const ChunkArgs& a, int id, float* lds) {
    const int hb = (a.H + kStepHeads - 1) / kStepHeads;
    const int h0 = id % hb * kStepHeads;
    const int chunk = id / hb % a.nc;
    const int seq = id / hb / a.nc;
    const int len = a.lengths ? a.lengths[seq] : a.T;
    if (len > a.T || chunk * Q >= len)
        return;
    const int heads = min(kStepHeads, a.H - h0);
    for (int i = threadIdx.x; i < Q * kStepHeads; i += blockDim.x) {   // [token][head] -> [head][token]
        const int t = chunk * Q + i / kStepHeads, k = i % kStepHeads;
        lds[k * (Q + 1) + i / kStepHeads] =
            t < len && k < heads ? a.p.dt[(static_cast<size_t>(seq) * a.T + t) * a.H + h0 + k] : 0.0f;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63;
    for (int k = threadIdx.x >> 6; k < heads; k += blockDim.x >> 6) {
        const int h = h0 + k;
        const float d = chunk * Q + lane < len
                            ? step_size(lds[k * (Q + 1) + lane] + (a.p.dt_bias ? a.p.dt_bias[h] : 0.0f)) : 0.0f;
        const double part = static_cast<double>(d) * static_cast<double>(rate2(a.p.A[h]));
        const double cum = wave_scan(part < kLeastDecay ? kLeastDecay : part, lane);
        const float high = static_cast<float>(cum);
        float* o = a.steps + ((static_cast<size_t>(seq) * a.H + h) * a.nc + chunk) * (3 * Q);
        o[lane] = d;
        o[Q + lane] = high;
        o[2 * Q + lane] = static_cast<float>(cum - static_cast<double>(high));
    }
}

// One workgroup of N / 16 waves per (sequence, group, chunk): a wave convolves 32
// of the group's 2 N channels.  B goes out straight from registers (a lane's
// runs of four tokens are the fragments' k order); C and the rows that G is
// formed from pass through LDS.  35 us at 32,768 tokens and one group (44 MB of
// fragments and inputs, 25 MB of steps), 68 us for eight prompts of up to 2,048
// tokens and 16 groups: bound by its chain of conv, scales, G and stores.
template <int N, typename Act, bool FINE>
__global__ __launch_bounds__(4 * N) void ssm_prep_kernel(ChunkArgs a, int prep_wgs) {
    using Sh = Shared<N, FINE>;
    constexpr int W = N / 16, KS = N / 16;
    constexpr int kRowHalfs = Q * N;   // one part of B's or C's rows, in fragment order
    extern __shared__ __align__(16) char pool[];
    if (static_cast<int>(blockIdx.x) >= prep_wgs) {
        steps_part(a, blockIdx.x - prep_wgs, reinterpret_cast<float*>(pool));
        return;
    }
    const int chunk = blockIdx.x % a.nc;
    const int g = blockIdx.x / a.nc % a.G;
    const int seq = blockIdx.x / a.nc / a.G;
    const int len = a.lengths ? a.lengths[seq] : a.T;
    const int t0 = chunk * Q;
    if (len > a.T || t0 >= len)
        return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hi = lane >> 5, c = lane & 31;
    const int half = wave / (W / 2);   // 0: B, 1: C
    const int nb = wave % (W / 2);     // 32-channel block
    const int ch0 = a.H * a.P + half * a.G * N + g * N + nb * 32;

    constexpr int kTiles = FINE ? 0 : W * Tile<Act>::kBytes;   // fp32 reads x directly
    constexpr int kRows = (FINE ? 4 : 2) * kRowHalfs * 2;
    _Float16* rows = reinterpret_cast<_Float16*>(pool);         // [B, C][hi, lo][fragments]; after the tiles' use
    float* part = reinterpret_cast<float*>(pool + (kTiles > kRows ? kTiles : kRows));   // [wave][2][64]
    float* sc = part + W * 2 * Q;                                                       // [B, C][64]

    Taps<Act> taps;
    taps.load(static_cast<const Act*>(a.p.w), static_cast<const Act*>(a.p.bias), ch0 + c);
    const Act* xs = static_cast<const Act*>(a.p.x) + static_cast<size_t>(seq) * a.T * a.C + ch0;
    const Act* tail = static_cast<const Act*>(a.p.tail_in) + (static_cast<size_t>(seq) * a.C + ch0) * 4;
    float u[32];
    if constexpr (FINE) {
        float tw[4];
        Quad<Act>::to_float(Quad<Act>::load(tail + c * 4), tw);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float v[7];
#pragma unroll
            for (int e = 0; e < 7; ++e) {
                const int t = t0 + 8 * r + 4 * hi + e - 3;
                const float x = xs[static_cast<size_t>(max(0, min(t, len - 1))) * a.C + c];
                v[e] = t >= 0 ? x : t == -1 ? tw[3] : t == -2 ? tw[2] : tw[1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float win[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
                u[4 * r + i] = conv_bias_silu(taps.w, win, taps.bias);
            }
        }
    } else {
        Stream<Act> in = make_stream(reinterpret_cast<Act*>(pool + wave * Tile<Act>::kBytes), xs, a.C, len, lane);
        in.load(t0);
        in.begin(tail, t0);
        in.store();
        wave_sync();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float v[4];
            conv_run(in.tile, taps, r, lane, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[4 * r + i] = v[i];
        }
    }
    if (t0 + Q > len) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
            u[k] = t0 + 8 * (k / 4) + 4 * hi + k % 4 < len ? u[k] : 0.0f;
    }
    // each token's row of B and of C is brought to [4, 8): |G| <= 64 N stays in range
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m[i] = row_max(u[4 * r + i]);
        if ((lane & 15) == 0)
            *reinterpret_cast<float4*>(part + (wave * 2 + ((lane >> 4) & 1)) * Q + 8 * r + 4 * hi) =
                make_float4(m[0], m[1], m[2], m[3]);
    }
    __syncthreads();
    _Float16* o = a.shared + ((static_cast<size_t>(seq) * a.G + g) * a.nc + chunk) * Sh::kHalfs;
    for (int i = threadIdx.x; i < 2 * Q; i += 4 * N) {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k)
            m = fmaxf(m, part[(i / Q * W + k) * Q + i % Q]);
        const float s = pow2_to<2, kMostBC>(m);
        sc[i] = s;
        reinterpret_cast<float*>(o + Sh::kFrags * 512)[i] = inverse_pow2(s);
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 s = *reinterpret_cast<const float4*>(sc + half * Q + 16 * ks + 8 * q + 4 * hi);
            const float ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[4 * q + i] = u[8 * ks + 4 * q + i] * ss[i];
        }
        h8 fh, fl;
        split8(v, fh, fl);
        if (half == 0) {
            st_frag(o, Sh::kB + nb * 4 + ks, lane, fh);
            st_frag(o, Sh::kBl + nb * 4 + ks, lane, fl);
        }
        // entry n of token t in fragment order of the rows
        const int n = nb * 32 + c;
        const int at = (n / 16 * 64 + ((n >> 2) & 1) * 32) * 8 + ((n >> 3) & 1) * 4 + (n & 3);
        _Float16* row = rows + half * (FINE ? 2 : 1) * kRowHalfs;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = 16 * ks + kperm(hi, e);
            const int pos = (t >> 5) * (KS * 512) + (t & 31) * 8 + at;
            row[pos] = fh[e];
            if (FINE)
                row[kRowHalfs + pos] = fl[e];
        }
    }
    __syncthreads();
    const _Float16* Br = rows;
    const _Float16* Cr = rows + (FINE ? 2 : 1) * kRowHalfs;
    for (int f = wave; f < Sh::CF; f += W) {
        st_frag(o, Sh::kC + f, lane, ld_frag(Cr, f, lane));
        if (FINE)
            st_frag(o, Sh::kCl + f, lane, ld_frag(Cr + kRowHalfs, f, lane));
    }
    // G transposed (rows j, columns i): its accumulators are the rows-i fragments
    for (int tile = wave; tile < 3; tile += W) {
        const int it = tile == 0 ? 0 : 1, jt = tile == 2 ? 1 : 0;
        f16v acc = zero16();
#pragma unroll 4
        for (int ks = 0; ks < KS; ++ks) {
            const h8 bh = ld_frag(Br, jt * KS + ks, lane), ch = ld_frag(Cr, it * KS + ks, lane);
            acc = mma(bh, ch, acc);
            if (FINE) {
                acc = mma(bh, ld_frag(Cr + kRowHalfs, it * KS + ks, lane), acc);
                acc = mma(ld_frag(Br + kRowHalfs, jt * KS + ks, lane), ch, acc);
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

template <int N, typename Act, bool FINE>
constexpr size_t prep_lds() {
    constexpr size_t tiles = FINE ? 0 : N / 16 * Tile<Act>::kBytes, rows = (FINE ? 4 : 2) * Q * N * 2;
    constexpr size_t prep = (tiles > rows ? tiles : rows) + N / 16 * 2 * Q * 4 + 2 * Q * 4;
    constexpr size_t steps = kStepHeads * (Q + 1) * 4;
    return prep > steps ? prep : steps;
}

// ------------------------------------------------------------ chunks

// Convolved x of one (sequence, head, chunk, 32 rows), as the output pass takes
// it.  bf16: four fragments in fp16 (k: tokens, columns: rows of the state), in a
// scale per row that follows them.  fp32: the lane's 32 values, four at a time.
template <bool FINE>
struct Conv {
    static constexpr size_t kBytes = FINE ? 64 * 32 * 4 : 4 * 1024 + 32 * 4;
};

// Which work is this workgroup's, and its place in memory; false: none.
struct Place {
    int g, h, seg, seq, len, ch0, ch1, last;
    size_t head;
};
__device__ __forceinline__ bool place(const ChunkArgs& a, bool report, Place& w, int heads = 1, int head = 0) {
    // workgroup -> (sequence, segment, group), heads of the group: all heads that
    // read the same fragments on one XCD (workgroups go to the eight in turn)
    const int rep = a.H / a.G / heads;
    int set, member;
    if (a.by_xcd) {
        set = blockIdx.x / 8 / rep * 8 + blockIdx.x % 8;
        member = blockIdx.x / 8 % rep;
    } else {
        set = blockIdx.x / rep;
        member = blockIdx.x % rep;
    }
    if (set >= a.B * a.segs * a.G)
        return false;
    w.g = set % a.G;
    w.h = (w.g * rep + member) * heads + head;
    w.seg = set / a.G % a.segs;
    w.seq = set / a.G / a.segs;
    w.head = static_cast<size_t>(w.seq) * a.H + w.h;
    w.len = a.lengths ? a.lengths[w.seq] : a.T;
    const bool bad = w.len < 0 || w.len > a.T;
    if (report && a.status && w.h == 0 && w.seg == 0 && threadIdx.x == 0)
        a.status[w.seq] = bad ? GDN_ERR_INDEX : GDN_OK;
    if (bad)
        return false;
    w.last = (w.len + Q - 1) / Q;
    w.ch0 = w.seg * a.chunks_per_seg;
    w.ch1 = min(w.ch0 + a.chunks_per_seg, w.last);
    return w.ch0 < w.ch1;
}

// The state, transposed: S[nt][v] is entry 32 nt + 8 (v / 4) + 4 hi + v % 4 of the
// lane's row; `row` points at entry 4 hi.
template <int NT>
__device__ __forceinline__ void load_state(f16v (&S)[NT], const float* row) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 v = *reinterpret_cast<const float4*>(row + 32 * nt + 8 * q);
            S[nt][4 * q] = v.x;
            S[nt][4 * q + 1] = v.y;
            S[nt][4 * q + 2] = v.z;
            S[nt][4 * q + 3] = v.w;
        }
}
template <int NT>
__device__ __forceinline__ void store_state(const f16v (&S)[NT], float out, float* row) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(row + 32 * nt + 8 * q) =
                make_float4(S[nt][4 * q] * out, S[nt][4 * q + 1] * out, S[nt][4 * q + 2] * out, S[nt][4 * q + 3] * out);
}
template <int NT>
__device__ __forceinline__ float state_max(const f16v (&S)[NT]) {
    float m = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            m = fmaxf(m, fabsf(S[nt][v]));
    return fmaxf(m, __shfl_xor(m, 32));
}

// Fragment f of M . G from G's; cH, cL: c per token.
template <typename Sh, bool FINE>
__device__ __forceinline__ void decayed_g(h8 gh, h8 gl, int f, const float* cH, const float* cL, int lane, h8& mh,
                                          h8& ml) {
    const int hi = lane >> 5, c = lane & 31;
    const int it = f >= 2, ks = it ? f - 2 : f;
    const float ci = cH[32 * it + c];
    const float li = FINE ? cL[32 * it + c] : 0.0f;
    float m[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = 16 * ks + 8 * q + 4 * hi;
        const float4 cj = *reinterpret_cast<const float4*>(cH + j);
        const float4 lj = FINE ? *reinterpret_cast<const float4*>(cL + j) : float4{};
        const float cc[4] = {cj.x, cj.y, cj.z, cj.w}, ll[4] = {lj.x, lj.y, lj.z, lj.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float arg = ci - cc[e];
            float gv = static_cast<float>(gh[4 * q + e]);
            if (FINE) {
                arg += li - ll[e];
                gv += static_cast<float>(gl[4 * q + e]);
            }
            m[4 * q + e] = j + e <= 32 * it + c ? gv * __builtin_amdgcn_exp2f(arg) : 0.0f;
        }
    }
    parts8<FINE>(m, mh, ml);
}

// The head's left factors of a chunk, [M . G | C], into LDS: each wave builds the fragments wave, wave + waves, ..., BATCH of them
// loaded at a time, the first batch well before it is needed.
template <int N, bool FINE, int BATCH>
struct Left {
    using Sh = Shared<N, FINE>;
    static constexpr int AF = Sh::GF + Sh::CF;
    h8 fh[BATCH], fl[BATCH];

    __device__ void load(const _Float16* sh, int f0, int waves, int lane) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int f = min(f0 + k * waves, AF - 1);   // always something: a value kept from before costs registers
            fh[k] = ld_frag(sh, f < Sh::GF ? Sh::kG + f : Sh::kC + f - Sh::GF, lane);
            if (FINE)
                fl[k] = ld_frag(sh, f < Sh::GF ? Sh::kGl + f : Sh::kCl + f - Sh::GF, lane);
        }
    }
    // cH, cL: c per token.  The first batch is loaded.
    __device__ void build(const _Float16* sh, _Float16* L, const float* cH, const float* cL, int wave, int waves,
                          int lane) {
        for (int f0 = wave; f0 < AF; f0 += BATCH * waves) {
            if (f0 != wave)
                load(sh, f0, waves, lane);
            phase();
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int f = f0 + k * waves;
                if (f >= AF)
                    break;
                h8 mh, ml;
                if (f < Sh::GF) {
                    decayed_g<Sh, FINE>(fh[k], fl[k], f, cH, cL, lane, mh, ml);
                } else {
                    mh = fh[k];
                    ml = fl[k];
                }
                st_frag(L, f, lane, mh);
                if (FINE)
                    st_frag(L, AF + f, lane, ml);
            }
        }
    }
};

// Y += C' S0^T, the state scaled by `scale` into fp16.  Ch, Cl: C's fragments.
template <int N, bool FINE>
__device__ __forceinline__ void state_product(f16v (&Y)[2], const f16v (&S)[N / 32], float scale, const _Float16* Ch,
                                              const _Float16* Cl, int lane) {
    constexpr int KS = N / 16;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = S[ks / 2][8 * (ks % 2) + e] * scale;
        h8 bh, bl;
        parts8<FINE>(v, bh, bl);
#pragma unroll
        for (int it = 0; it < 2; ++it) {
            const h8 ah = ld_frag(Ch, it * KS + ks, lane);
            Y[it] = mma(ah, bh, Y[it]);
            if (FINE) {
                Y[it] = mma(ah, bl, Y[it]);
                Y[it] = mma(ld_frag(Cl, it * KS + ks, lane), bh, Y[it]);
            }
        }
        if (ks % 4 == 3)
            phase();
    }
}
// Y += (M . G) X'
template <int N, bool FINE>
__device__ __forceinline__ void chunk_product(f16v (&Y)[2], const h8 (&xh)[4], const h8 (&xl)[4], const _Float16* L,
                                              int lane) {
    using Sh = Shared<N, FINE>;
    constexpr int AF = Sh::GF + Sh::CF;
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
}

// A chunk's gate z, 32 tokens at a time.  Where there are registers it is asked for
// before the state's update and ahead of the far loads (N = 256, 2 x 4,000 tokens:
// 234 -> 217 us).
template <typename Act>
struct Gate {
    using Tl = Tile<Act>;
    static constexpr int kHalf = Tl::kPerRow / 2;
    u4 raw[2][kHalf];
    __device__ void load(int it, const Act* z, int pitch, int rows, int lane) {
        const int urow = lane / Tl::kPerRow, ucol = lane % Tl::kPerRow * Tl::kUnit;
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
            const int r = min(32 * it + urow + k * Tl::kRowStep, rows - 1);
            raw[it][k] =
                at<const u4>(z, static_cast<uint32_t>(r * pitch + ucol) * static_cast<uint32_t>(sizeof(Act)));
        }
    }
};

// Y * (rows' factors fS) * back, gated, to y: 32 tokens at a time through the
// wave's tile, 16 bytes per store.  y and z point at the chunk's first token and
// the wave's first channel.  AHEAD: the gate is loaded already.
template <bool AHEAD, typename Act>
__device__ __forceinline__ void store_y(const f16v (&Y)[2], const float* fS, float back, float* tile, Act* y,
                                        const Act* z, const Gate<Act>& gate, int pitch, int rows, int lane) {
    using Tl = Tile<Act>;
    constexpr int kHalf = Tl::kPerRow / 2;
    constexpr uint32_t kSize = sizeof(Act);
    const int hi = lane >> 5, c = lane & 31;
    const int urow = lane / Tl::kPerRow, ucol = lane % Tl::kPerRow * Tl::kUnit;
    union Unit {
        u4 raw;
        Act v[Tl::kUnit];
    };
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        Gate<Act> own;
        if (!AHEAD && z)
            own.load(it, z, pitch, rows, lane);
        phase();
        wave_sync();   // what was in the tile is read
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 Sc = *reinterpret_cast<const float4*>(fS + 32 * it + 8 * q + 4 * hi);
            const float sc[4] = {Sc.x, Sc.y, Sc.z, Sc.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tile[(8 * q + 4 * hi + i) * Tl::kPitch + c] = Y[it][4 * q + i] * (sc[i] * back);
        }
        wave_sync();
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
            const int r = urow + k * Tl::kRowStep;
            float o[Tl::kUnit];
#pragma unroll
            for (int q = 0; q < Tl::kUnit / 4; ++q) {
                const float4 v = *reinterpret_cast<const float4*>(tile + r * Tl::kPitch + ucol + 4 * q);
                o[4 * q] = v.x;
                o[4 * q + 1] = v.y;
                o[4 * q + 2] = v.z;
                o[4 * q + 3] = v.w;
            }
            Unit yu, zu;
            if (z) {
                zu.raw = (AHEAD ? gate : own).raw[it][k];
#pragma unroll
                for (int e = 0; e < Tl::kUnit; ++e)
                    o[e] *= silu(widen(zu.v[e]));
            }
#pragma unroll
            for (int e = 0; e < Tl::kUnit; ++e)
                narrow(o[e], yu.v[e]);
            if (32 * it + r < rows)
                at<u4>(y, static_cast<uint32_t>((32 * it + r) * pitch + ucol) * kSize) = yu.raw;
        }
    }
}

// The conv tails after the prompt, by the workgroups of its last chunk: a wave
// its own channels, and the group's first head B's and C's.
template <typename Act>
__device__ void write_tails(const ChunkArgs& a, const Place& w, int wave, int N, int lane) {
    const int col0 = w.h * a.P + wave * 32;
    auto put = [&](int ch) {
        Act* tp = static_cast<Act*>(a.p.tail_out) + (static_cast<size_t>(w.seq) * a.C + ch) * 4;
        const Act* xs = static_cast<const Act*>(a.p.x) + static_cast<size_t>(w.seq) * a.T * a.C + ch;
        typename Quad<Act>::raw t = Quad<Act>::load(tp);
#pragma unroll
        for (int j = 4; j >= 1; --j)
            if (w.len >= j)
                t = Quad<Act>::push(t, xs[static_cast<size_t>(w.len - j) * a.C]);
        Quad<Act>::store(tp, t);
    };
    if (lane < 32)
        put(col0 + lane);
    if (w.h % (a.H / a.G) == 0)
        for (int i = wave * 64 + lane; i < 2 * N; i += a.P * 2)
            put(a.H * a.P + (i < N ? 0 : a.G * N) + w.g * N + i % N);
}

// B's fragments, a k-step at a time: the caller loads the first, update() each
// other one as the products before it are issued.
template <int N, bool FINE>
struct BSteps {
    using Sh = Shared<N, FINE>;
    static constexpr int NT = N / 32;
    h8 h[NT], l[NT];
    __device__ void load(const _Float16* sh, int ks, int lane) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            h[nt] = ld_frag(sh, Sh::kB + nt * 4 + ks, lane);
            l[nt] = ld_frag(sh, Sh::kBl + nt * 4 + ks, lane);
        }
    }
    // S = keep S + X''^T B
    __device__ void update(f16v (&S)[NT], float keep, const h8 (&wh)[4], const h8 (&wl)[4], const _Float16* sh,
                           int lane) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                S[nt][v] *= keep;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            // parts outside, tiles inside: products of one accumulator do not follow one another
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                S[nt] = mma(h[nt], wh[ks], S[nt]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                S[nt] = mma(h[nt], wl[ks], S[nt]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                S[nt] = mma(l[nt], wh[ks], S[nt]);
            if (ks < 3) {
                load(sh, ks + 1, lane);
                phase();
            }
        }
    }
};

// The same fragments, loaded once by the four waves of a workgroup and passed on
// through LDS.
template <int N, bool FINE>
struct BShare {
    using Sh = Shared<N, FINE>;
    static constexpr int NT = N / 32, PER = 2 * Sh::BF / 4;
    static constexpr size_t kBytes = 2 * Sh::BF * 1024;
    h8 r[PER];
    __device__ void load(const _Float16* sh, int wave, int lane) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            r[k] = ld_frag(sh, Sh::kB + wave * PER + k, lane);
    }
    __device__ void store(_Float16* B, int wave, int lane) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            st_frag(B, wave * PER + k, lane, r[k]);
    }
    // beside(ks, m): vector work that fills the time of k-step ks's m-th product (-1: before the first).
    template <typename F>
    __device__ static void update(f16v (&S)[NT], float keep, const h8 (&wh)[4], const h8 (&wl)[4], const _Float16* B,
                                  int lane, F&& beside) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                S[nt][v] *= keep;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            h8 h[NT], l[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                h[nt] = ld_frag(B, nt * 4 + ks, lane);
            beside(ks, -1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                S[nt] = mma(h[nt], wh[ks], S[nt]);
                l[nt] = ld_frag(B, Sh::BF + nt * 4 + ks, lane);
                beside(ks, nt);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                S[nt] = mma(h[nt], wl[ks], S[nt]);
                beside(ks, NT + nt);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                S[nt] = mma(l[nt], wh[ks], S[nt]);
                beside(ks, 2 * NT + nt);
            }
            phase();
        }
    }
};

// Each segment's own state from zero, the state's products in two fp16 parts, and
// the convolved x for the output pass.  One wave per 32 rows of the state; a
// workgroup is one head's waves, which share nothing, or (SHARE) four waves of
// heads of one group, which load B's fragments once for all and convolve the next
// chunk between the products of this one.  32,768 tokens of 64 heads, P = 64,
// N = 128: 193 us at the fastest of 20 calls back to back (221 in the median, as
// the clock falls), 537 MB in and out at 2.8 TB/s.  What is left: the matrix
// products (41 us at the peak rate), and on the vector unit conv, SiLU, X''s scale
// and the fp16 parts, 670 instructions per chunk and wave (75 us).  The last chunk
// has a copy of its own: with a branch for it the loop spills 104 registers.
template <int N, typename Act, bool FINE, bool SHARE>
__global__ __launch_bounds__(256, N > 128 ? 1 : 2) void ssm_state_kernel(ChunkArgs a) {
    using Sh = Shared<N, FINE>;
    using Tl = Tile<Act>;
    constexpr int NT = N / 32;
    extern __shared__ __align__(16) char pool[];   // [waves][tile, factors], then B's fragments
    const int lane = threadIdx.x & 63;
    const int wave_wg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hi = lane >> 5, c = lane & 31;
    const int waves = a.P / 32;
    const int wave = SHARE ? wave_wg % waves : wave_wg;
    Place w;
    if (!place(a, false, w, SHARE ? 4 / waves : 1, SHARE ? wave_wg / waves : 0))
        return;
    const int col0 = w.h * a.P + wave * 32;
    char* mine = pool + wave_wg * (Tl::kBytes + Q * 4);
    _Float16* Bs = reinterpret_cast<_Float16*>(pool + 4 * (Tl::kBytes + Q * 4));
    float* fF = reinterpret_cast<float*>(mine + Tl::kBytes);   // d * 2^-s_B * 2^(c_last - c), X'' over x
    const float* steps = a.steps + w.head * a.nc * (3 * Q);
    const _Float16* shared0 = a.shared + (static_cast<size_t>(w.seq) * a.G + w.g) * a.nc * Sh::kHalfs;
    char* conv = a.conv + (w.head * a.nc * waves + wave) * Conv<FINE>::kBytes;

    Taps<Act> taps;
    taps.load(static_cast<const Act*>(a.p.w), static_cast<const Act*>(a.p.bias), col0 + c);
    Stream<Act> in = make_stream(reinterpret_cast<Act*>(mine),
                                 static_cast<const Act*>(a.p.x) + static_cast<size_t>(w.seq) * a.T * a.C + col0, a.C,
                                 w.len, lane);
    float st_d, st_h, st_l, st_b;   // the chunk's step, c and scale (one token per lane)
    auto load_steps = [&](int ch) {
        const float* st = steps + static_cast<size_t>(ch) * (3 * Q);
        st_d = st[lane];
        st_h = st[Q + lane];
        st_l = st[2 * Q + lane];
        st_b = reinterpret_cast<const float*>(shared0 + ch * Sh::kHalfs + Sh::kFrags * 512)[lane];
    };
    std::conditional_t<SHARE, BShare<N, FINE>, BSteps<N, FINE>> B;
    f16v S[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        S[nt] = zero16();
    float unit = 1.0f;   // S holds the state times this, at most `most`
    float most = 0.0f;
    double seg_sum = 0.0;
    float xc[32], mx = 0.0f;   // the chunk's convolved x and its largest magnitude
    auto conv_runs = [&](int r0, int r1) {
#pragma unroll
        for (int r = r0; r < r1; ++r) {
            float v[4];
            conv_run(in.tile, taps, r, lane, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xc[4 * r + i] = v[i];
                mx = fmaxf(mx, fabsf(v[i]));
                pin(xc[4 * r + i]);
            }
            pin(mx);
        }
    };
    in.load(w.ch0 * Q);
    load_steps(w.ch0);
    in.begin(static_cast<const Act*>(a.p.tail_in) + (static_cast<size_t>(w.seq) * a.C + col0) * 4, w.ch0 * Q);
    in.store();
    wave_sync();
    in.load(min(w.ch0 + 1, w.ch1 - 1) * Q);
    B.load(shared0 + w.ch0 * Sh::kHalfs, SHARE ? wave_wg : 0, lane);
    phase();
#pragma unroll
    for (int r = 0; r < 8; r += 2) {
        conv_runs(r, r + 2);
        phase();
    }

    const auto step = [&](int ch, auto last) {
        constexpr bool more = !decltype(last)::value;   // a chunk follows
        const _Float16* sh = shared0 + ch * Sh::kHalfs;
        const float th = __shfl(st_h, 63), tl = __shfl(st_l, 63);
        seg_sum += static_cast<double>(th) + static_cast<double>(tl);
        fF[lane] = st_d * st_b * __builtin_amdgcn_exp2f((th - st_h) + (tl - st_l));
        const float decay = __builtin_amdgcn_exp2f(th + tl);
        if (more)
            in.save(Q);
        wave_sync();
        if (more)
            load_steps(ch + 1);
        mx = fmaxf(mx, __shfl_xor(mx, 32));

        // x is left behind, and becomes X'' in its place
        const float sx = pow2_to<8, kMostX>(mx);
        char* to = conv + static_cast<size_t>(ch) * waves * Conv<FINE>::kBytes;
        float mw = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if constexpr (FINE) {
#pragma unroll
                for (int r = 2 * ks; r < 2 * ks + 2; ++r)
                    reinterpret_cast<float4*>(to)[r * 64 + lane] =
                        make_float4(xc[4 * r], xc[4 * r + 1], xc[4 * r + 2], xc[4 * r + 3]);
            } else {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[e] = xc[8 * ks + e] * sx;
                st_frag(reinterpret_cast<_Float16*>(to), ks, lane, half8(u));
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 F = *reinterpret_cast<const float4*>(fF + 16 * ks + 8 * q + 4 * hi);
                const float ff[4] = {F.x, F.y, F.z, F.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = 8 * ks + 4 * q + i;
                    xc[e] *= ff[i];
                    mw = fmaxf(mw, fabsf(xc[e]));
                    pin(xc[e]);
                }
            }
            pin(mw);
            phase();
        }
        // X'' in a scale of its own: a row's largest decides, wherever in the chunk decays and inputs leave it
        mw = fmaxf(mw, __shfl_xor(mw, 32));
        const float s2 = unit_for(mw, unit, decay * most);
        h8 wh[4], wl[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = xc[8 * ks + e] * s2;
            split8(v, wh[ks], wl[ks]);
            pin(wh[ks]);
            pin(wl[ks]);
        }
        phase();
        if (!FINE && lane < 32)
            reinterpret_cast<float*>(to + 4096)[lane] = inverse_pow2(sx);
        const float keep = decay * (s2 * inverse_pow2(unit));
        unit = s2;
        most = __builtin_fmaf(keep, most, kMostUpdate);
        // the next chunk's rows into the tile; its conv runs beside the products of this one
        if (more)
            in.store();
        mx = 0.0f;
        Run<Act> run[2];
        const auto beside = [&](int ks, int m) {   // two runs' eight values over 3 NT products
            if (!more)
                return;
            if (m < 0) {
                run[0].load(in.tile, 2 * ks, lane);
                run[1].load(in.tile, 2 * ks + 1, lane);
                return;
            }
#pragma unroll
            for (int j = 8 * m / (3 * NT); j < 8 * (m + 1) / (3 * NT); ++j) {
                const int e = 8 * ks + j;
                xc[e] = run[j / 4].out(taps, j % 4);
                mx = fmaxf(mx, fabsf(xc[e]));
                pin(xc[e]);
                pin(mx);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (SHARE) {
            __syncthreads();   // the last chunk's fragments are used
            B.store(Bs, wave_wg, lane);
            __syncthreads();
            if (more)
                B.load(sh + Sh::kHalfs, wave_wg, lane);
        }
        wave_sync();
        if (more)
            in.load(min(ch + 2, w.ch1 - 1) * Q);
        phase();
        if constexpr (SHARE) {
            B.update(S, keep, wh, wl, Bs, lane, beside);
        } else {
            B.update(S, keep, wh, wl, sh, lane);
            if (more) {
                B.load(sh + Sh::kHalfs, 0, lane);
                phase();
#pragma unroll
                for (int r = 0; r < 8; r += 2) {
                    conv_runs(r, r + 2);
                    phase();
                }
            }
        }
        phase();
    };
    for (int ch = w.ch0; ch + 1 < w.ch1; ++ch)
        step(ch, std::false_type{});
    step(w.ch1 - 1, std::true_type{});
    store_state(S, inverse_pow2(unit),
                a.seg_state + (w.head * a.segs + w.seg) * a.P * N + static_cast<size_t>(wave * 32 + c) * N + 4 * hi);
    if (wave == 0 && lane == 0)
        a.seg_decay[w.head * a.segs + w.seg] = static_cast<float>(seg_sum);
}

// Each segment's own state becomes the state that enters it; the state itself
// goes to the end of the prompt.  One thread per four entries; 16 us for 32
// segments' states of 64 heads of 64 x 128 (67 MB each way), 26 us for eight
// prompts of 48 heads of 128 x 128.
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
    constexpr int U = 8;   // segments in flight
    for (int k0 = 0; k0 < n; k0 += U) {
        float4 own[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k0 + k < n)
                own[k] = sg[static_cast<int64_t>(k0 + k) * quads];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k0 + k < n) {
                sg[static_cast<int64_t>(k0 + k) * quads] = s;
                const float d = __builtin_amdgcn_exp2f(dec[k0 + k]);
                s = make_float4(__builtin_fmaf(d, s.x, own[k].x), __builtin_fmaf(d, s.y, own[k].y),
                                __builtin_fmaf(d, s.z, own[k].z), __builtin_fmaf(d, s.w, own[k].w));
            }
    }
    *st = s;
}

// C's and B's fragments (the high parts) for the output pass: loaded once by the
// waves of a workgroup and passed on through LDS, C first.
template <int N>
struct Common {
    using Sh = Shared<N, false>;
    static constexpr int NT = N / 32, kFrags = Sh::CF + Sh::BF, PER = kFrags / 4;   // PER: of a wave of four
    h8 r[PER];
    __device__ void load(const _Float16* sh, int f0, int step, int lane) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int f = min(f0 + k * step, kFrags - 1);
            r[k] = ld_frag(sh, f < Sh::CF ? Sh::kC + f : Sh::kB + f - Sh::CF, lane);
        }
    }
    // The first fragments are loaded; fewer than four waves take more than one turn.
    __device__ void store(_Float16* to, const _Float16* sh, int wave, int waves, int lane) {
        for (int f0 = wave; f0 < kFrags; f0 += PER * waves) {
            if (f0 != wave)
                load(sh, f0, waves, lane);
#pragma unroll
            for (int k = 0; k < PER; ++k)
                st_frag(to, f0 + k * waves, lane, r[k]);
        }
    }
    // S = keep S + X''^T B
    __device__ static void update(f16v (&S)[NT], float keep, const h8 (&wh)[4], const _Float16* B, int lane) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                S[nt][v] *= keep;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                S[nt] = mma(ld_frag(B, nt * 4 + ks, lane), wh[ks], S[nt]);
    }
};

// A wave's part of the output pass's LDS.
constexpr size_t out_wave_bytes() { return Tile<uint16_t>::kBytes + 5 * Q * 4 + Q * 2; }

// The output pass over segments of bf16 activations, from the states that enter
// them and the convolved x.  Its own state only serves outputs that are rounded
// to bf16: one fp16 part each, X' formed in packed fp16 and X'', which needs a
// scale of its own, in fp32 (in fp16 too, 219 instead of 224 us, it would be gone
// behind a decay of 2^-25).  One wave per 32 rows of the state; a workgroup is
// `heads` heads of one group, which share C's and B's fragments, and a head's waves
// its M . G.  The decay of the state that enters is put on the products' rows, so
// that C needs none of its own.  32,768 tokens of 64 heads, P = 64, N = 128: 224 us
// at the fastest of 20 calls back to back (255 in the median), 537 MB in and out at
// 2.4 TB/s, bound like the state pass by its chain of small phases per chunk.
template <int N>
__global__ __launch_bounds__(256, N > 128 ? 1 : 2) void ssm_out_kernel(ChunkArgs a, int heads) {
    using Act = uint16_t;
    using Sh = Shared<N, false>;
    using Tl = Tile<Act>;
    constexpr int NT = N / 32;
    using Cs = Common<N>;
    // [C and B][heads][M . G][waves][tile, factors]
    extern __shared__ __align__(16) char pool[];
    const int lane = threadIdx.x & 63;
    const int wave_wg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hi = lane >> 5, c = lane & 31;
    const int waves = a.P / 32, waves_wg = heads * waves;
    const int wave = wave_wg % waves;
    Place w;
    if (!place(a, true, w, heads, wave_wg / waves))
        return;
    const int col0 = w.h * a.P + wave * 32;
    _Float16* common = reinterpret_cast<_Float16*>(pool);
    _Float16* L = common + (Cs::kFrags + wave_wg / waves * Sh::GF) * 512;
    char* mine = pool + (Cs::kFrags + heads * Sh::GF) * 1024 + wave_wg * out_wave_bytes();
    float* yt = reinterpret_cast<float*>(mine);
    float* fS = reinterpret_cast<float*>(mine + Tl::kBytes);   // 2^-s_C
    float* fK = fS + Q;                                        // D * s_F * 2^s_C
    float* fH = fS + 2 * Q;                                    // c, high part
    float* fE = fS + 3 * Q;                                    // 2^c
    float* fW = fS + 4 * Q;                                    // d * 2^-s_B * 2^(c_last - c), X'' over x
    _Float16* fF = reinterpret_cast<_Float16*>(fS + 5 * Q);    // d * 2^-s_B * s_F
    const float skip = a.p.D ? a.p.D[w.h] : 0.0f;
    const float* steps = a.steps + w.head * a.nc * (3 * Q);
    const _Float16* shared0 = a.shared + (static_cast<size_t>(w.seq) * a.G + w.g) * a.nc * Sh::kHalfs;
    const char* conv = a.conv + (w.head * a.nc * waves + wave) * Conv<false>::kBytes;
    const size_t yrow = static_cast<size_t>(a.H) * a.P;

    float st_d, st_h, st_l, st_b, st_c, st_x;
    h8 xq[4];
    auto load_chunk = [&](int ch) {
        const float* st = steps + static_cast<size_t>(ch) * (3 * Q);
        st_d = st[lane];
        st_h = st[Q + lane];
        st_l = st[2 * Q + lane];
        const float* sc = reinterpret_cast<const float*>(shared0 + ch * Sh::kHalfs + Sh::kFrags * 512);
        st_b = sc[lane];
        st_c = sc[Q + lane];
        const char* from = conv + static_cast<size_t>(ch) * waves * Conv<false>::kBytes;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            xq[ks] = ld_frag(reinterpret_cast<const _Float16*>(from), ks, lane);
        st_x = reinterpret_cast<const float*>(from + 4096)[c];
    };
    Cs cb;
    constexpr int kG = 3;   // fragments of G in flight
    h8 gf[kG];
    auto load_g = [&](const _Float16* sh, int f0) {
#pragma unroll
        for (int k = 0; k < kG; ++k)
            gf[k] = ld_frag(sh, Sh::kG + min(f0 + k * waves, Sh::GF - 1), lane);
    };
    f16v S[NT];
    float unit = 1.0f;
    load_chunk(w.ch0);
    load_state(S, a.seg_state + (w.head * a.segs + w.seg) * a.P * N + static_cast<size_t>(wave * 32 + c) * N + 4 * hi);

    for (int ch = w.ch0; ch < w.ch1; ++ch) {
        const _Float16* sh = shared0 + ch * Sh::kHalfs;
        const int next = min(ch + 1, w.ch1 - 1);
        load_g(sh, wave);
        cb.load(sh, wave_wg, waves_wg, lane);
        const float th = __shfl(st_h, 63), tl = __shfl(st_l, 63);
        const float F = st_d * st_b;
        const float sF = pow2_to<0, kMostF>(wave_max(F));
        const float cs = st_x;
        fF[lane] = static_cast<_Float16>(F * sF);
        fW[lane] = F * __builtin_amdgcn_exp2f((th - st_h) + (tl - st_l));
        fS[lane] = st_c;
        fK[lane] = skip * sF * inverse_pow2(st_c);
        fH[lane] = st_h;
        fE[lane] = __builtin_amdgcn_exp2f(st_h + st_l);
        const float decay = __builtin_amdgcn_exp2f(th + tl);
        wave_sync();
        // X' in units of s_F / cs; x itself is taken up by Y below.  X'' in fp32, then in a scale of its own: a row's
        // largest decides, wherever in the chunk decays and inputs leave it
        const float ux = sF * inverse_pow2(cs);
        h8 xh[4], wh[4];
        float xw[32], mw = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            typedef _Float16 h4 __attribute__((ext_vector_type(4)));
            h8 f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const h4 f4_ = *reinterpret_cast<const h4*>(fF + 16 * ks + 8 * q + 4 * hi);
                const float4 W = *reinterpret_cast<const float4*>(fW + 16 * ks + 8 * q + 4 * hi);
                const float ww[4] = {W.x, W.y, W.z, W.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = 8 * ks + 4 * q + i;
                    f[4 * q + i] = f4_[i];
                    xw[e] = __builtin_fmaf(static_cast<float>(xq[ks][4 * q + i]), ww[i], 0.0f);
                    mw = fmaxf(mw, fabsf(xw[e]));
                    pin(xw[e]);
                }
            }
            pin(mw);
            xh[ks] = xq[ks] * f;
            pin(xh[ks]);
        }
        mw = fmaxf(mw, __shfl_xor(mw, 32));
        const float largest = state_max(S);
        const float uw = unit_for(mw * cs, unit, decay * largest);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf(xw[8 * ks + e], uw * cs, 0.0f);
            wh[ks] = half8(v);
            pin(wh[ks]);
        }
        for (int f0 = wave; f0 < Sh::GF; f0 += kG * waves) {
            if (f0 != wave)
                load_g(sh, f0);
#pragma unroll
            for (int k = 0; k < kG; ++k)
                if (f0 + k * waves < Sh::GF) {
                    h8 mh, ml;
                    decayed_g<Sh, false>(gf[k], gf[k], f0 + k * waves, fH, fH, lane, mh, ml);
                    st_frag(L, f0 + k * waves, lane, mh);
                }
        }
        cb.store(common, sh, wave_wg, waves_wg, lane);
        const float ss = pow2_to<8, kMostS>(largest);   // on top of `unit`
        phase();
        __syncthreads();
        f16v Y[2] = {zero16(), zero16()};
        state_product<N, false>(Y, S, ss, common, common, lane);
        // to X's unit and the tokens' decays, and D x
        const float ratio = ux * (inverse_pow2(ss) * inverse_pow2(unit));
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 K = *reinterpret_cast<const float4*>(fK + 32 * it + 8 * q + 4 * hi);
                const float4 E = *reinterpret_cast<const float4*>(fE + 32 * it + 8 * q + 4 * hi);
                const float kk[4] = {K.x, K.y, K.z, K.w}, ee[4] = {E.x, E.y, E.z, E.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y = __builtin_fmaf(static_cast<float>(xq[2 * it + q / 2][4 * (q % 2) + i]), kk[i],
                                             Y[it][4 * q + i] * (ratio * ee[i]));
                    pin(y);
                    Y[it][4 * q + i] = y;
                }
            }
        phase();
        // loads are counted in the order of issue: those that are waited for first go first
        const size_t y0 = (static_cast<size_t>(w.seq) * a.T + ch * Q) * yrow + col0;
        const Act* z = a.p.z ? static_cast<const Act*>(a.p.z) + y0 : nullptr;
        Gate<Act> gate;
        if (z) {
            gate.load(0, z, static_cast<int>(yrow), w.len - ch * Q, lane);
            gate.load(1, z, static_cast<int>(yrow), w.len - ch * Q, lane);
        }
        load_chunk(next);
        phase();
        chunk_product<N, false>(Y, xh, xh, L, lane);
        phase();
        if (ch + 1 < w.ch1) {
            Cs::update(S, decay * (uw * inverse_pow2(unit)), wh, common + Sh::CF * 512, lane);
            unit = uw;
        }
        phase();
        store_y<true>(Y, fS, inverse_pow2(ux), yt, static_cast<Act*>(a.p.y) + y0, z, gate, static_cast<int>(yrow),
                      w.len - ch * Q, lane);
        __syncthreads();   // what the waves share is rewritten by the next chunk
        wave_sync();       // and so are tile and factors
    }
    if (w.ch1 == w.last)
        write_tails<Act>(a, w, wave, N, lane);
}

// A wave's part of its LDS, less the left factor.
template <typename Act>
constexpr size_t chunk_wave_bytes() { return Tile<Act>::kBytes + 7 * Q * 4; }

// The output pass that also carries the state (one segment), or takes the state
// and the convolved x of segments in fp32.  One workgroup per (sequence, segment,
// head), one wave per 32 rows of the state; the waves share the left factors.  The
// decay of the state that enters goes to the products' rows in fp32, not to C.
// 16 prompts of 1,024 tokens, 64 heads, P = 64, N = 128: 212 to 218 us a call with
// prep (348 MB with the states, 1.6 TB/s), bound by its chain per chunk at two waves per SIMD; fp32,
// 2 x 1,003 tokens in segments: 28 us, one wave per SIMD.  One scale per row for X',
// X'' and the state took 202 us, but what is large in one takes bits from another.
// Spills: 3 registers at N = 128, 12 to 24 at N = 256.
template <int N, typename Act, bool FINE, bool SPLIT>
__global__ __launch_bounds__(256, N > 128 || FINE ? 1 : 2) void ssm_chunk_kernel(ChunkArgs a) {
    using Sh = Shared<N, FINE>;
    using Tl = Tile<Act>;
    constexpr int NT = N / 32;
    static_assert(FINE || !SPLIT, "bf16 segments are ssm_out_kernel's");
    extern __shared__ __align__(16) char pool[];   // [waves][tile, factors], then the left factor
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hi = lane >> 5, c = lane & 31;
    const int waves = a.P / 32;
    Place w;
    if (!place(a, true, w))
        return;
    const int col0 = w.h * a.P + wave * 32;
    char* mine = pool + wave * chunk_wave_bytes<Act>();
    float* yt = reinterpret_cast<float*>(mine);
    float* fF = reinterpret_cast<float*>(mine + Tl::kBytes);   // d * 2^-s_B, X' over x
    float* fW = fF + Q;                                        // the same times 2^(c_last - c), X'' over x
    float* fS = fF + 2 * Q;                                    // 2^-s_C
    float* fK = fF + 3 * Q;                                    // D * 2^s_C
    float* fH = fF + 4 * Q;                                    // c, high and low part
    float* fL = fF + 5 * Q;
    float* fE = fF + 6 * Q;                                    // 2^c
    _Float16* L = reinterpret_cast<_Float16*>(pool + waves * chunk_wave_bytes<Act>());
    const float skip = a.p.D ? a.p.D[w.h] : 0.0f;
    const float* steps = a.steps + w.head * a.nc * (3 * Q);
    const _Float16* shared0 = a.shared + (static_cast<size_t>(w.seq) * a.G + w.g) * a.nc * Sh::kHalfs;
    const char* conv = a.conv + (w.head * a.nc * waves + wave) * Conv<FINE>::kBytes;
    const size_t yrow = static_cast<size_t>(a.H) * a.P;

    Taps<Act> taps;
    taps.load(static_cast<const Act*>(a.p.w), static_cast<const Act*>(a.p.bias), col0 + c);
    Stream<Act> in = make_stream(reinterpret_cast<Act*>(mine),
                                 static_cast<const Act*>(a.p.x) + static_cast<size_t>(w.seq) * a.T * a.C + col0, a.C,
                                 w.len, lane);
    float st_d, st_h, st_l, st_b, st_c;
    auto load_steps = [&](int ch) {
        const float* st = steps + static_cast<size_t>(ch) * (3 * Q);
        st_d = st[lane];
        st_h = st[Q + lane];
        st_l = st[2 * Q + lane];
        const float* sc = reinterpret_cast<const float*>(shared0 + ch * Sh::kHalfs + Sh::kFrags * 512);
        st_b = sc[lane];
        st_c = sc[Q + lane];
    };
    BSteps<N, FINE> B;
    Left<N, FINE, (FINE ? 4 : 8)> left;
    f16v S[NT];
    float unit = 1.0f;
    const size_t row_off = static_cast<size_t>(wave * 32 + c) * N + 4 * hi;
    float* state_row = SPLIT ? a.seg_state + (w.head * a.segs + w.seg) * a.P * N + row_off
                             : a.p.state + w.head * a.P * N + row_off;
    load_steps(w.ch0);
    float4 xn[8];   // the next chunk's convolved x (with the gate's early loads fp32, 2 x 5,000 tokens: 155 -> 134 us)
    auto load_x = [&](int ch) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
            xn[r] = reinterpret_cast<const float4*>(conv + static_cast<size_t>(ch) * waves *
                                                               Conv<FINE>::kBytes)[r * 64 + lane];
    };
    if constexpr (SPLIT) {
        load_x(w.ch0);
    } else {
        in.load(w.ch0 * Q);
        in.begin(static_cast<const Act*>(a.p.tail_in) + (static_cast<size_t>(w.seq) * a.C + col0) * 4, w.ch0 * Q);
    }
    load_state(S, state_row);

    for (int ch = w.ch0; ch < w.ch1; ++ch) {
        const _Float16* sh = shared0 + ch * Sh::kHalfs;
        const int next = min(ch + 1, w.ch1 - 1);
        if constexpr (!SPLIT)
            in.store();
        const float th = __shfl(st_h, 63), tl = __shfl(st_l, 63);
        const float F = st_d * st_b;
        fF[lane] = F;
        fW[lane] = F * __builtin_amdgcn_exp2f((th - st_h) + (tl - st_l));
        fS[lane] = st_c;
        fK[lane] = skip * inverse_pow2(st_c);
        fH[lane] = st_h;
        fL[lane] = st_l;
        fE[lane] = __builtin_amdgcn_exp2f(st_h + st_l);
        const float decay = __builtin_amdgcn_exp2f(th + tl);
        wave_sync();
        if constexpr (!SPLIT)
            in.load(next * Q);
        load_steps(next);

        float xc[32];
        float mx = 0.0f, mF = 0.0f, mW = 0.0f;   // largest of x, X' and X''
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float v[4];
            if constexpr (SPLIT) {
                v[0] = xn[r].x, v[1] = xn[r].y, v[2] = xn[r].z, v[3] = xn[r].w;
            } else {
                conv_run(in.tile, taps, r, lane, v);
            }
            const float4 F4 = *reinterpret_cast<const float4*>(fF + 8 * r + 4 * hi);
            const float4 W4 = *reinterpret_cast<const float4*>(fW + 8 * r + 4 * hi);
            const float ff[4] = {F4.x, F4.y, F4.z, F4.w}, ww[4] = {W4.x, W4.y, W4.z, W4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xc[4 * r + i] = v[i];
                mx = fmaxf(mx, fabsf(v[i]));
                mF = fmaxf(mF, fabsf(v[i] * ff[i]));
                mW = fmaxf(mW, fabsf(v[i] * ww[i]));
                pin(xc[4 * r + i]);
            }
            pin(mx);
            pin(mF);
            pin(mW);
            if (!SPLIT && r % 2)
                phase();
        }
        if constexpr (SPLIT)
            load_x(next);
        else
            in.save(Q);
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        mF = fmaxf(mF, __shfl_xor(mF, 32));
        mW = fmaxf(mW, __shfl_xor(mW, 32));
        // on their way while X' is formed (16 x 500 tokens of 32 heads, N = 256: 216 -> 208 us, fp32 303 -> 287)
        left.load(sh, wave, waves, lane);
        // X' and with it Y, X'' and with it the next state, and the state that enters, each in a scale of its own: what
        // is large in one does not take bits from another.  D x stays within fp32's range in Y's.
        const float largest = state_max(S);
        const float u = fminf(unit_for(mF, unit, largest), pow2_to<60, 100>(mx));
        const float uw = unit_for(mW, unit, decay * largest);
        const float ss = pow2_to<8, kMostS>(largest);   // on top of `unit`
        // X'' and X' as fragments; x itself for D x (for bf16 outputs in fp16)
        const float sx = FINE ? 1.0f : pow2_to<8, kMostX>(mx);
        h8 wh[4], wl[4], xh[4], xl[4], xq[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            float xw[8], xp[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 F4 = *reinterpret_cast<const float4*>(fF + 16 * ks + 8 * q + 4 * hi);
                const float4 W4 = *reinterpret_cast<const float4*>(fW + 16 * ks + 8 * q + 4 * hi);
                const float ff[4] = {F4.x, F4.y, F4.z, F4.w}, ww[4] = {W4.x, W4.y, W4.z, W4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = xc[8 * ks + 4 * q + i];
                    xw[4 * q + i] = x * ww[i] * uw;
                    xp[4 * q + i] = x * ff[i] * u;
                }
            }
            if constexpr (!FINE) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = xc[8 * ks + e] * sx;
                xq[ks] = half8(v);
                pin(xq[ks]);
            }
            split8(xw, wh[ks], wl[ks]);
            parts8<FINE>(xp, xh[ks], xl[ks]);
            pin(wh[ks]);
            pin(wl[ks]);
            pin(xh[ks]);
            if (FINE)
                pin(xl[ks]);
            phase();
        }
        left.build(sh, L, fH, fL, wave, waves, lane);
        phase();
        __syncthreads();
        const bool update = !SPLIT || ch + 1 < w.ch1;
        constexpr int GF = Sh::GF, AF = Sh::GF + Sh::CF;
        f16v Y[2] = {zero16(), zero16()};
        state_product<N, FINE>(Y, S, ss, L + GF * 512, L + (AF + GF) * 512, lane);
        // to Y's unit and the tokens' decays, and D x
        const float ratio = u * (inverse_pow2(ss) * inverse_pow2(unit)), ux = u * inverse_pow2(sx);
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 K = *reinterpret_cast<const float4*>(fK + 32 * it + 8 * q + 4 * hi);
                const float4 E = *reinterpret_cast<const float4*>(fE + 32 * it + 8 * q + 4 * hi);
                const float kk[4] = {K.x, K.y, K.z, K.w}, ee[4] = {E.x, E.y, E.z, E.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = FINE ? xc[16 * it + 4 * q + i]
                                         : static_cast<float>(xq[2 * it + q / 2][4 * (q % 2) + i]);
                    float y = __builtin_fmaf(x * ux, kk[i], Y[it][4 * q + i] * (ratio * ee[i]));
                    pin(y);
                    Y[it][4 * q + i] = y;
                }
            }
        chunk_product<N, FINE>(Y, xh, xl, L, lane);
        if (update)
            B.load(sh, 0, lane);
        const size_t y0 = (static_cast<size_t>(w.seq) * a.T + ch * Q) * yrow + col0;
        const Act* z = a.p.z ? static_cast<const Act*>(a.p.z) + y0 : nullptr;
        Gate<Act> gate;   // ahead where there are registers for it
        if (FINE && z) {
            gate.load(0, z, static_cast<int>(yrow), w.len - ch * Q, lane);
            gate.load(1, z, static_cast<int>(yrow), w.len - ch * Q, lane);
        }
        phase();
        if (update) {
            B.update(S, decay * (uw * inverse_pow2(unit)), wh, wl, sh, lane);
            unit = uw;
        }
        phase();
        store_y<FINE>(Y, fS, inverse_pow2(u), yt, static_cast<Act*>(a.p.y) + y0, z, gate, static_cast<int>(yrow),
                      w.len - ch * Q, lane);
        __syncthreads();   // the left factor is rewritten by the next chunk
        wave_sync();       // and so are tile and factors
    }
    if constexpr (!SPLIT)
        store_state(S, inverse_pow2(unit), state_row);
    if (w.ch1 == w.last)
        write_tails<Act>(a, w, wave, N, lane);
}

// ------------------------------------------------------------ host

// Segments per sequence: as many as fill the chip once, which is two waves per
// SIMD, or one where a wave needs more than 256 registers (N = 256, fp32).  One
// 64-head prompt of 32,768 tokens: 463 us at 2,048 waves, 478 at half as many
// again, 477 at 4,096; N = 256 (32 heads, 4,096 tokens) 100 us at 1,024, 127 at
// 1,536 and 129 at 2,048.  Prompts of given lengths end at different times and take
// twice as many (eight of up to 2,048 tokens: 313 against 335 us).  A segment has at
// least two chunks, in fp32 one (64 heads, 512 tokens: 54 us with four, 43 with two,
// 47 with one; fp32, 32 heads, 256 tokens: 53, 45 and 36 us).
// Returns the number before it is evened out, which does not fall as T grows.
static int segments(const SsmGeo& g, int T, bool ragged, int& segs, int& per) {
    const int nc = (T + Q - 1) / Q;
    const int64_t waves = static_cast<int64_t>(g.B) * g.H * (g.P / 32);
    const int64_t fill = (g.N > 128 || !g.bf16 ? 1024 : 2048) * (ragged ? 2 : 1);
    const int64_t want = (fill + waves - 1) / waves;
    const int most = std::max(1, nc / (g.bf16 ? 2 : 1));
    const int limit = static_cast<int>(std::min<int64_t>(want, most));
    per = (nc + limit - 1) / limit;
    segs = (nc + per - 1) / per;
    return limit;
}

static size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

static size_t shared_halfs(const SsmGeo& g) {
    const bool fine = !g.bf16;
    switch (g.N) {
        case 32: return fine ? Shared<32, true>::kHalfs : Shared<32, false>::kHalfs;
        case 64: return fine ? Shared<64, true>::kHalfs : Shared<64, false>::kHalfs;
        case 128: return fine ? Shared<128, true>::kHalfs : Shared<128, false>::kHalfs;
        default: return fine ? Shared<256, true>::kHalfs : Shared<256, false>::kHalfs;
    }
}

// The workspace: fragments, steps, and with segments their states, decays and the convolved x.  It has room for the
// segments' limit, so that one sized for a prompt serves every shorter one.
static size_t carve(const SsmGeo& g, int T, bool ragged, char* base, ChunkArgs* a) {
    int segs, per;
    const int limit = segments(g, T, ragged, segs, per);
    const size_t nc = (T + Q - 1) / Q, BH = static_cast<size_t>(g.B) * g.H;
    size_t n = 0;
    auto take = [&](size_t bytes) {
        const size_t at = n;
        n += up256(bytes);
        return at;
    };
    const size_t shared = take(static_cast<size_t>(g.B) * g.G * nc * shared_halfs(g) * sizeof(_Float16));
    const size_t steps = take(BH * nc * (3 * Q) * sizeof(float));
    size_t state = 0, decay = 0, conv = 0;
    if (limit > 1) {
        state = take(BH * limit * g.P * g.N * sizeof(float));
        decay = take(BH * limit * sizeof(float));
        conv = take(BH * nc * (g.P / 32) * (g.bf16 ? Conv<false>::kBytes : Conv<true>::kBytes));
    }
    if (a) {
        a->shared = reinterpret_cast<_Float16*>(base + shared);
        a->steps = reinterpret_cast<float*>(base + steps);
        a->seg_state = reinterpret_cast<float*>(base + state);   // read with segments only, like the next two
        a->seg_decay = reinterpret_cast<float*>(base + decay);
        a->conv = base + conv;
        a->nc = static_cast<int>(nc);
        a->segs = segs;
        a->chunks_per_seg = per;
    }
    return n;
}

size_t chunked_ws_bytes(const SsmGeo& g, int T) {
    return std::max(carve(g, T, false, nullptr, nullptr), carve(g, T, true, nullptr, nullptr));
}

// A launch that may need more than 64 KB of LDS.
template <typename... Args>
static hipError_t launch_lds(void (*kernel)(Args...), dim3 grid, dim3 block, size_t lds, hipStream_t s, Args... args) {
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(kernel, grid, block, lds, s, args...);
    return hipGetLastError();
}

template <int N, typename Act, bool FINE>
static hipError_t chunked_cfg(const SsmGeo& g, const SsmArgs& p, int T, const int32_t* lengths, int32_t* status,
                              void* ws, hipStream_t s) {
    ChunkArgs a{};
    a.p = p;
    a.lengths = lengths;
    a.status = status;
    a.T = T, a.B = g.B, a.H = g.H, a.G = g.G, a.P = g.P, a.C = g.C;
    carve(g, T, lengths != nullptr, static_cast<char*>(ws), &a);
    // by XCD where the sets of heads come out even over the eight, or nearly
    const int64_t sets = static_cast<int64_t>(g.B) * g.G * a.segs;
    a.by_xcd = sets % 8 == 0 || sets >= 64;

    const int prep_wgs = g.B * g.G * a.nc;
    const int step_wgs = g.B * a.nc * ((g.H + kStepHeads - 1) / kStepHeads);
    hipError_t e = launch_lds(ssm_prep_kernel<N, Act, FINE>, dim3(prep_wgs + step_wgs), dim3(4 * N),
                              prep_lds<N, Act, FINE>(), s, a, prep_wgs);
    if (e != hipSuccess)
        return e;
    const int waves = g.P / 32;
    const int64_t wgs = (a.by_xcd ? (sets + 7) / 8 * 8 : sets) * (g.H / g.G);
    const dim3 grid(static_cast<unsigned>(wgs)), block(64 * waves);
    constexpr int kTile = Tile<Act>::kBytes;
    constexpr int kLeft = (FINE ? 2 : 1) * (Shared<N, FINE>::GF + Shared<N, FINE>::CF) * 1024;
    const size_t lds_chunk = waves * chunk_wave_bytes<Act>() + kLeft;
    if (a.segs == 1)
        return launch_lds(ssm_chunk_kernel<N, Act, FINE, false>, grid, block, lds_chunk, s, a);
    // Heads of a workgroup, which share what does not depend on the head.  It pays
    // where the chip is more than half full, at two waves per SIMD or one (64 heads:
    // 32,768 tokens 592 -> 463 us, 4 x 4,096 318 -> 248; N = 256, 32 heads, 4,096
    // tokens 121 -> 100); below that barriers and coarser workgroups cost more than the
    // loads that they save (512 tokens 43.0 -> 45.6 us), except for heads of 128 rows,
    // whose workgroups stay as they are (eight prompts of up to 2,048: 327 -> 313 us).
    const int rep = g.H / g.G;
    const bool share = waves == 4 || wgs * waves > (N > 128 ? 512 : 1024);
    const int heads = !share ? 1 : rep % (4 / waves) == 0 ? 4 / waves : waves == 1 && rep % 2 == 0 ? 2 : 1;
    if (share && heads * waves == 4)
        e = launch_lds(ssm_state_kernel<N, Act, FINE, true>, dim3(static_cast<unsigned>(wgs / heads)), dim3(256),
                       4 * (kTile + Q * 4) + BShare<N, FINE>::kBytes, s, a);
    else
        e = launch_lds(ssm_state_kernel<N, Act, FINE, false>, grid, block, waves * (kTile + Q * 4), s, a);
    if (e != hipSuccess)
        return e;
    const int quads = g.P * N / 4;
    const int64_t threads = static_cast<int64_t>(g.B) * g.H * quads;
    hipLaunchKernelGGL(ssm_join_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, s, a, quads);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    if constexpr (FINE)
        return launch_lds(ssm_chunk_kernel<N, Act, true, true>, grid, block, lds_chunk, s, a);
    else
        return launch_lds(ssm_out_kernel<N>, dim3(static_cast<unsigned>(wgs / heads)), dim3(64 * heads * waves),
                          heads * waves * out_wave_bytes() + (Common<N>::kFrags + heads * Shared<N, false>::GF) * 1024,
                          s, a, heads);
}

hipError_t launch_ssm_chunked(const SsmGeo& g, const SsmArgs& p, int T, const int32_t* lengths, int32_t* status,
                              void* ws, hipStream_t s) {
    switch (g.N) {
        case 32: return g.bf16 ? chunked_cfg<32, uint16_t, false>(g, p, T, lengths, status, ws, s)
                               : chunked_cfg<32, float, true>(g, p, T, lengths, status, ws, s);
        case 64: return g.bf16 ? chunked_cfg<64, uint16_t, false>(g, p, T, lengths, status, ws, s)
                               : chunked_cfg<64, float, true>(g, p, T, lengths, status, ws, s);
        case 128: return g.bf16 ? chunked_cfg<128, uint16_t, false>(g, p, T, lengths, status, ws, s)
                                : chunked_cfg<128, float, true>(g, p, T, lengths, status, ws, s);
        default: return g.bf16 ? chunked_cfg<256, uint16_t, false>(g, p, T, lengths, status, ws, s)
                               : chunked_cfg<256, float, true>(g, p, T, lengths, status, ws, s);
    }
}

}  // namespace ssm
}  // namespace gdn
