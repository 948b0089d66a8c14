// gdn_beam.hip -- beam search over recurrent states: the selection over beams
// and vocabulary, and the move of the beams' states.
//
// Selection.  Candidate (k, v) of a sequence has the value
//   score_k + (l_kv - m_k) - log sum_v exp(l_kv - m_k),   m_k = max_v l_kv
// and the S best of the K*V are wanted, ties to the lowest k*V + v.  Within a
// beam the order is the order of its logits, so one pass over the logits keeps
// the running maximum, the sum of exponentials and the S best (logit, index)
// pairs of each span of a row; a second, small launch joins the spans.
//   scan  one wave per span of a row, four neighbouring spans to a workgroup.  The
//         largest of each lane's first logits gives a bound that at least S of the
//         row's logits reach (the S-th largest of the workgroup's 256, by
//         bisection with ballots); what reaches it goes to the wave's buffer in
//         LDS.  A buffer that fills is cut to its S best, and its bound raised, by
//         the same bisection.  64 x 8 rows of 128,000 bf16 logits: 33.5 us, 3.1 TB/s
//         of what it reads (rows of ended beams are not); what is beside the
//         stream is the running sum's exponentials and the upkeep of the bound.
//   join  one workgroup per sequence: each beam's sum over the spans in fp64,
//         then the S best of the spans' entries by their fp64 value; 5 to 7 us, a
//         chain of loads, sums and three barriers.  Candidates are counted against
//         each other: where nearly all are equal (rows of one value, K * S = 2,048)
//         that is 8,192 against 8,192.
// Keys (ordered logit bits, complement of the index) are unique, so the result
// does not depend on the order in which spans or waves finish.
#include <algorithm>

#include "gdn.h"
#include "gdn_core.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace beam {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSpans = 64;

// A masked or broken logit (NaN) counts as -inf and +inf as the largest finite
// value, so that a row keeps a finite maximum.
__device__ __forceinline__ float clean(float v) {
    return v == v ? (v > __FLT_MAX__ ? __FLT_MAX__ : v) : -__builtin_inff();
}
// Order-preserving map of a clean float to an unsigned integer (0 is below all); -0 is 0.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u));
}

// The next float above a finite or -inf v.
__device__ __forceinline__ float next_up(float v) {
    const int u = __float_as_int(v + 0.0f);
    return __int_as_float(u < 0 ? u - 1 : u + 1);
}

template <typename Act>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int E = 8, kLowBits = 16;   // ordered keys of bf16 differ above bit 15 only
    typedef uint32_t raw __attribute__((ext_vector_type(4)));
    // the bf16 value whose key has the high bits of T
    __device__ static float value(uint32_t T) {
        return __uint_as_float(__float_as_uint(unordered(T)) & 0xFFFF0000u);
    }
    __device__ static raw load(const uint16_t* p) { return __builtin_nontemporal_load(reinterpret_cast<const raw*>(p)); }
    __device__ static void unpack(raw r, float (&v)[8]) {
        // cleaned only where some lane has an exponent of all ones (packed magnitudes' largest)
        typedef uint16_t us2 __attribute__((ext_vector_type(2)));
        us2 big = __builtin_bit_cast(us2, r[0] & 0x7FFF7FFFu);
#pragma unroll
        for (int j = 1; j < 4; ++j)
            big = __builtin_elementwise_max(big, __builtin_bit_cast(us2, r[j] & 0x7FFF7FFFu));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(r[j] << 16);
            v[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
        }
        if (__ballot(big.x >= 0x7F80 || big.y >= 0x7F80)) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = clean(v[e]);
        }
    }
};
template <>
struct Vec<float> {
    static constexpr int E = 4, kLowBits = 0;
    typedef nt4 raw;
    __device__ static float value(uint32_t T) { return unordered(T); }
    __device__ static raw load(const float* p) { return __builtin_nontemporal_load(reinterpret_cast<const nt4*>(p)); }
    __device__ static void unpack(raw r, float (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = clean(r[j]);
    }
};

constexpr uint32_t kLeast = 0x00800000u;   // the key after -inf's
constexpr uint32_t kMost = 0xFF7FFFFFu;    // the largest finite value's

// A T (a multiple of 2^low) that at least `want` of the lanes' values reach, and
// the largest such if more do; 0 if fewer have a value.  A lane has R values,
// value(0) .. value(R - 1).  With all 32 bits to go through, the search ends where
// exactly `want` reach it (scan of fp32 logits 12.0 -> 11.3 us); with fewer the
// largest T is worth its last steps (the join 7.0 -> 7.8 us without them).  It
// does not end below kLeast: what lies under -inf's key is no logit's, and read as a
// float it would be a NaN, which nothing reaches.
template <int R, typename F>
__device__ __forceinline__ uint32_t reached_by(int want, int low, F&& value) {
    uint32_t T = 0;
#pragma unroll 1
    for (int b = 31; b >= low; --b) {
        const uint32_t c = T | 1u << b;
        int n = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
            n += __popcll(__ballot(value(r) >= c));
        if (n >= want)
            T = c;
        if (low == 0 && n == want && T >= kLeast)
            break;
    }
    return T;
}

// A span's maximum and its sum of exponentials.  The sum is kept in fp64: what
// it loses shifts every candidate of the beam against the other beams'.
struct alignas(16) Part {
    double s;
    float m, unused;
};

// Running maximum and sum of exponentials of one lane.  The maximum moves rarely
// after the first vectors, so it is moved only where some lane's does.
struct Sum {
    float m = -__builtin_inff(), ref = 0.0f, s = 0.0f;   // ref: m, or 0 before there is one
    template <int E>
    __device__ float add(const float (&v)[E]) {
        float top = v[0];
#pragma unroll
        for (int e = 1; e < E; ++e)
            top = fmaxf(top, v[e]);
        if (__ballot(top > m)) {
            const float now = fmaxf(m, top);
            const float to = now == -__builtin_inff() ? 0.0f : now;
            s *= __builtin_amdgcn_exp2f((m - to) * kLog2e);   // m = -inf: s is 0
            m = now;
            ref = to;
        }
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = __builtin_amdgcn_exp2f((v[e] - ref) * kLog2e);
#pragma unroll
        for (int w = E / 2; w >= 1; w /= 2)
#pragma unroll
            for (int e = 0; e < w; ++e)
                x[e] += x[e + w];
        s += x[0];
        return top;
    }
};

// Reductions over a wave by DPP within rows of 16 lanes, then over the four rows.
template <int CTRL>
__device__ __forceinline__ double dpp_move64(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    const int lo = static_cast<int>(u), hi = static_cast<int>(u >> 32);
    const uint32_t l = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, lo, CTRL, 0xF, 0xF, false));
    const uint32_t h = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, hi, CTRL, 0xF, 0xF, false));
    return __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(h) << 32 | l));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    const uint32_t l = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), lane));
    const uint32_t h = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane));
    return __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(h) << 32 | l));
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_move64<0xB1>(v);
    v += dpp_move64<0x4E>(v);
    v += dpp_move64<0x141>(v);
    v += dpp_move64<0x140>(v);
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_move<0xB1>(v));
    v = fmaxf(v, dpp_move<0x4E>(v));
    v = fmaxf(v, dpp_move<0x141>(v));
    v = fmaxf(v, dpp_move<0x140>(v));
    float r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        r[k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * k));
    return fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
}

// A buffer is cut when S + kKeep entries are passed: often enough to raise the
// bound while the row's best are still being found.
constexpr int kKeep = 48;
constexpr int kBuf = 64 + kKeep + 64 * 8;   // and what one more step can add
constexpr int kRounds = (kBuf + 63) / 64;

// Cuts a wave's n buffered keys to the S best (n > S), R per lane at most.
// Returns an ordered logit that they reach and no other does, but for equals of it.
template <int R>
__device__ __forceinline__ uint32_t cut_rounds(uint2* buf, int n, int S, int low, int lane) {
    uint32_t hi[R], lo[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint2 k = r * 64 + lane < n ? buf[r * 64 + lane] : make_uint2(0, 0);
        hi[r] = k.x;
        lo[r] = k.y;
    }
    uint32_t T = reached_by<R>(S, low, [&](int r) { return hi[r]; });
    uint32_t top = T + ((1u << low) - 1);   // the values of this step: T .. top
    if (top == kMost) {   // two values: bf16's largest, T, and what +inf counts as
        int inf = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
            inf += __popcll(__ballot(hi[r] == kMost));
        (inf >= S ? T : top) = inf >= S ? kMost : T;
    }
    int above = 0, reach = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        above += __popcll(__ballot(hi[r] > top));
        reach += __popcll(__ballot(hi[r] >= T && hi[r] != 0));
    }
    uint32_t I = 0;   // among equals the lowest indices: the largest complements
    if (reach > S)
        I = reached_by<R>(S - above, 0, [&](int r) { return hi[r] >= T && hi[r] <= top ? lo[r] : 0u; });
    int at = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool take = hi[r] != 0 && (hi[r] > top || (hi[r] >= T && lo[r] >= I));
        const uint64_t mask = __ballot(take);
        if (take)
            buf[at + lanes_below(mask)] = make_uint2(hi[r], lo[r]);
        at += __popcll(mask);
    }
    return T;
}
// Few entries are the rule; the general form is kept out of the way (and called,
// not inlined: a span is short, and code that is fetched once costs like data).
__device__ __attribute__((noinline)) uint32_t cut_many(uint2* buf, int n, int S, int low, int lane) {
    return cut_rounds<kRounds>(buf, n, S, low, lane);
}
__device__ __forceinline__ uint32_t cut(uint2* buf, int n, int S, int low, int lane) {
    return n <= 2 * kWave ? cut_rounds<2>(buf, n, S, low, lane) : cut_many(buf, n, S, low, lane);
}

template <typename Act>
__global__ __launch_bounds__(256) void beam_scan_kernel(const Act* __restrict__ logits,
                                                        const float* __restrict__ scores,
                                                        const uint8_t* __restrict__ finished, int64_t pitch, int V,
                                                        int S, int spans, Part* __restrict__ sums,
                                                        uint2* __restrict__ keys) {
    using Vc = Vec<Act>;
    constexpr int E = Vc::E, U = 64 / E;   // vectors per lane that the first bound comes from
    __shared__ uint2 bufs[4][kBuf];
    __shared__ uint32_t tops[4 * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    uint2* buf = bufs[wave];
    const int wgs = spans / 4;
    const int64_t row = blockIdx.x / wgs;
    const int span = (blockIdx.x % wgs) * 4 + wave;
    // a beam that has ended, or does not exist, has no use for its logits
    if ((finished && finished[row]) || clean(scores[row]) == -__builtin_inff())
        return;
    const Act* p = logits + row * pitch;
    // logits before the first 16-byte boundary of the row, and whole vectors after it
    int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / static_cast<int>(sizeof(Act));
    head = head < V ? head : V;
    const int nvec = (V - head) / E;
    const int per = (nvec + spans - 1) / spans;
    const int v0 = span * per < nvec ? span * per : nvec;
    const int v1 = v0 + per < nvec ? v0 + per : nvec;
    const Act* body = p + head;

    Sum sum;
    int n = 0;                         // entries in the buffer
    float bound = -__builtin_inff();   // logits that reach it are wanted
    bool above = false;                // it is already past the value that S entries reach
    // the lanes of `in` whose logit is wanted
    auto wanted = [&](float v, uint64_t in) { return __ballot(v >= bound) & in; };
    auto put = [&](float v, uint32_t index, uint64_t mask) {
        if (__builtin_amdgcn_inverse_ballot_w64(mask))
            buf[n + lanes_below(mask)] = make_uint2(ordered(v), ~index);
        n += __popcll(mask);
    };
    // Between steps, with S entries that reach the bound: later equals of it have
    // higher indices and are not wanted any more.
    auto pass = [&](float value) {
        bound = next_up(value);
        above = true;
    };
    auto trim = [&]() {
        if (n > S + kKeep) {
            pass(Vc::value(cut(buf, n, S, Vc::kLowBits, lane)));
            n = S;
        }
    };
    // the few logits before the vectors
    if (span == 0 && head > 0) {
        const bool in = lane < head;
        float v[1] = {in ? clean(widen(p[lane])) : -__builtin_inff()};
        sum.add(v);
        put(v[0], static_cast<uint32_t>(lane), __ballot(in));
    }
    typename Vc::raw raw[U];
    const int last = v1 - 1;
    // the first U vectors per lane, and the bound from the lanes' maxima of them
    float top = -__builtin_inff();
    if (v0 < v1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u] = Vc::load(body + static_cast<int64_t>(min(v0 + u * kWave + lane, last)) * E);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[E];
            Vc::unpack(raw[u], v);
#pragma unroll
            for (int e = 0; e < E; ++e)
                top = fmaxf(top, v0 + u * kWave + lane < v1 ? v[e] : -__builtin_inff());
        }
    }
    tops[threadIdx.x] = v0 + lane < v1 ? ordered(top) : 0;
    __syncthreads();
    uint32_t all[4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
        all[w] = tops[w * kWave + lane];
    const uint32_t T = reached_by<4>(S, Vc::kLowBits, [&](int w) { return all[w]; });
    if (T)
        bound = Vc::value(T);
    const int before = n;   // may be below the bound
    for (int j0 = v0; j0 < v1; j0 += U * kWave) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * kWave + lane;
            const bool in = j < v1;
            const uint64_t ins = __ballot(in);
            float v[E];
            Vc::unpack(raw[u], v);
            if (j0 + (U + u) * kWave < v1)   // the vector of the next round
                raw[u] = Vc::load(body + static_cast<int64_t>(min(j + U * kWave, last)) * E);
            if (j0 + u * kWave + kWave > v1) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    v[e] = in ? v[e] : -__builtin_inff();
            }
            if (wanted(sum.add(v), ins)) {
                uint64_t mask[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    mask[e] = wanted(v[e], ins);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (mask[e])
                        put(v[e], static_cast<uint32_t>(head + j * E + e), mask[e]);
                trim();
            }
        }
        if (!above && n - before >= S)
            pass(bound);
    }
    // and the few after them
    if (span == 0) {
        const int i = head + nvec * E + lane;
        const bool in = i < V;
        float v[1] = {in ? clean(widen(p[i])) : -__builtin_inff()};
        sum.add(v);
        put(v[0], static_cast<uint32_t>(i), wanted(v[0], __ballot(in)));
    }
    if (n > S) {
        cut(buf, n, S, Vc::kLowBits, lane);
        n = S;
    }
    // the wave's maximum and sum
    const float m = wave_max(sum.m);
    const float ref = m == -__builtin_inff() ? 0.0f : m;
    const double s =
        wave_sum(static_cast<double>(sum.s) * static_cast<double>(__builtin_amdgcn_exp2f((sum.m - ref) * kLog2e)));
    const int64_t slot = row * spans + span;
    if (lane == 0)
        sums[slot] = Part{s, m, 0.0f};
    if (lane < S)
        keys[slot * S + lane] = lane < n ? buf[lane] : make_uint2(0, 0);
}

// fp64 counterpart of the ordered map.
__device__ __forceinline__ uint64_t ordered64(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double unordered64(uint64_t o) {
    return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}
constexpr int kJoinWaves = 16;
constexpr int kMaxEntries = 8192;   // of one sequence, over beams and spans

// One workgroup per sequence.  Every entry is taken once, by one thread.  Each
// wave finds a bound that S of its threads' best reach; what reaches the largest
// of these bounds is gathered in LDS and each candidate counts those before it:
// that is its place.  R: entries per thread; 8, for K * S > 512, needs more than the
// 128 registers that 1,024 threads leave and spills 120 (one request of 32 beams,
// best 64 of 150,000 entries each: 145 us a call).
template <int R>
__global__ __launch_bounds__(64 * kJoinWaves) void beam_join_kernel(
    const Part* __restrict__ sums, const uint2* __restrict__ keys, const float* scores,
    const uint8_t* __restrict__ finished, int eos, int K, int V, int S, int spans, float* out_scores,
    int32_t* __restrict__ parent, int32_t* __restrict__ token) {
    // A beam's entry of logit l has the value sc + ((l - m) - logs).
    struct Beam {
        double sc, m, logs;
        int live, only_eos;   // live: its logits count; else at most `eos`, at sc
    };
    __shared__ Beam beams[GDN_MAX_BEAMS];
    __shared__ uint32_t bounds[kJoinWaves];
    __shared__ int count;
    extern __shared__ __align__(16) char pool[];
    uint64_t* cv = reinterpret_cast<uint64_t*>(pool);                 // the candidates' values, then
    uint32_t* ci = reinterpret_cast<uint32_t*>(cv + K * spans * S);   // their indices' complements, then
    int* places = reinterpret_cast<int*>(ci + K * spans * S);         // how many come before each
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = tid / kWave;
    const int64_t seq = blockIdx.x;
    const int n = spans * S, total = K * n;
    // entries are on their way while the beams' sums are formed
    uint2 q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = r * 64 * kJoinWaves + tid;
        q[r] = e < total ? keys[seq * total + e] : make_uint2(0, 0);
    }
    if (tid == 0)
        count = 0;
    for (int k = wave; k < K; k += kJoinWaves) {
        const int64_t row = seq * K + k;
        const float sc = clean(scores[row]) + 0.0f;
        const bool fin = finished && finished[row];
        const Part part = lane < spans ? sums[row * spans + lane] : Part{0.0, -__builtin_inff(), 0.0f};
        const float m = wave_max(part.m);
        const double s =
            wave_sum(part.m == -__builtin_inff() ? 0.0 : part.s * exp(static_cast<double>(part.m) - m));
        const bool none = sc == -__builtin_inff();
        if (lane == 0)
            beams[k] = Beam{sc, m, log(s), !fin && !none && m != -__builtin_inff(), fin && !none};
    }
    __syncthreads();
    uint64_t v[R];
    uint32_t i[R];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        v[r] = 0;
        i[r] = 0;
        const int e = r * 64 * kJoinWaves + tid;
        if (e < total) {
            const int k = e / n;
            const Beam& b = beams[k];
            const uint32_t flat0 = static_cast<uint32_t>(k) * static_cast<uint32_t>(V);
            if (b.live) {
                const double l = static_cast<double>(unordered(q[r].x));
                v[r] = q[r].x ? ordered64((b.sc + ((l - b.m) - b.logs)) + 0.0) : 0;
                i[r] = ~(flat0 + ~q[r].y);
            } else {
                // eos first where the beam has ended, then the lowest tokens at -inf, S in all
                const int o = e - k * n;
                const int t = b.only_eos ? (o == 0 ? eos : o - 1 < eos ? o - 1 : o) : o;
                v[r] = o >= S || t >= V ? 0 : ordered64(b.only_eos && o == 0 ? b.sc : -__builtin_inf());
                i[r] = ~(flat0 + static_cast<uint32_t>(t));
            }
        }
        const uint32_t h = static_cast<uint32_t>(v[r] >> 32);
        top = h > top ? h : top;
    }
    // sign, exponent and eight bits of the value are enough of a bound
    const uint32_t own = reached_by<1>(S, 12, [&](int) { return top; });
    if (lane == 0)
        bounds[wave] = own;
    __syncthreads();
    uint32_t bound = 0;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w)
        bound = bounds[w] > bound ? bounds[w] : bound;
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (v[r] && static_cast<uint32_t>(v[r] >> 32) >= bound) {
            const int at = atomicAdd(&count, 1);   // any order: places come from the keys
            cv[at] = v[r];
            ci[at] = i[r];
            places[at] = 0;
        }
    __syncthreads();
    // each candidate's place, counted by as many threads as there are for it (at least S candidates: a bound is
    // reached by S of a wave's, and every beam's spans hold the S best of its logits)
    const int c = max(count, 1);
    const int parts = c < 64 * kJoinWaves ? 64 * kJoinWaves / c : 1;
    for (int e = tid / parts; e < c; e += 64 * kJoinWaves) {
        const uint64_t val = cv[e];
        const uint32_t idx = ci[e];
        int before = 0;
#pragma unroll 4
        for (int o = tid % parts; o < c; o += parts)
            before += cv[o] > val || (cv[o] == val && ci[o] > idx);
        if (before)
            atomicAdd(&places[e], before);
    }
    __syncthreads();
    for (int e = tid; e < c; e += 64 * kJoinWaves) {
        const int place = places[e];
        if (place < S) {
            const uint64_t val = cv[e];
            const uint32_t flat = ~ci[e];
            out_scores[seq * S + place] = static_cast<float>(unordered64(val));
            parent[seq * S + place] = static_cast<int32_t>(flat / static_cast<uint32_t>(V));
            token[seq * S + place] = static_cast<int32_t>(flat % static_cast<uint32_t>(V));
        }
    }
}

// Spans per row: 4,096 waves over all rows, spans of at least 1,024 logits, at most
// one span per lane of a joining wave and kMaxEntries entries per sequence; a
// multiple of the four waves of a workgroup.  4,096 waves are what the bf16 scan has
// room for, four per SIMD (64 x 8 rows of 128,000: 41 us a call, 45 with 2,048, 42 to
// 44 with 8,192); the fp32 scan has room for three and loses little by it (the same
// rows, best 8: 61 us, 57.5 with a quarter fewer, 63 with 8,192).
static int spans_of(int B, int K, int V, int S) {
    const int64_t rows = static_cast<int64_t>(B) * K;
    int64_t n = std::min<int64_t>((4096 + rows - 1) / rows, (static_cast<int64_t>(V) + 1023) / 1024);
    n = std::min<int64_t>(n, 2048 / (K * S));   // at most two entries per joining thread, where four spans allow it
    return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 4) / 4 * 4, kMaxSpans));
}

// Reorder.  A thread owns one 16-byte unit of a sequence's state (or tail) in
// every slot of its group: it loads, for each slot that takes another's state,
// the unit from that slot's parent, and stores only after its last load.  No
// other thread touches those units, so the move is in place without a second
// copy of the states, and slots that keep their own state cost nothing.  Bound
// by HBM: the sources that move are read, the slots that move are written (8 x 4
// beams of 3.2 MB with parents drawn at random: 137 MB in 21.8 us).
template <int KM>
__global__ __launch_bounds__(256) void beam_reorder_kernel(float* __restrict__ S, float* __restrict__ T, int64_t su,
                                                           int64_t tu, int K, const int32_t* __restrict__ parent,
                                                           int32_t* __restrict__ status, int wgs) {
    const int64_t group = blockIdx.x / wgs;
    const int part = blockIdx.x % wgs;
    int32_t from[KM];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        from[k] = k < K ? parent[group * K + k] : k;
        bad |= k < K && (from[k] < 0 || from[k] >= K);
    }
    if (status && part == 0 && threadIdx.x == 0)
        status[group] = bad ? GDN_ERR_INDEX : GDN_OK;
    const int64_t u = static_cast<int64_t>(part) * 256 + threadIdx.x;
    if (bad || u >= su + tu)
        return;
    float* base = u < su ? S + (group * K * su + u) * 4 : T + (group * K * tu + (u - su)) * 4;
    const int64_t step = (u < su ? su : tu) * 4;
    nt4 v[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k)
        v[k] = from[k] != k ? *reinterpret_cast<const nt4*>(base + from[k] * step) : nt4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (from[k] != k)
            __builtin_nontemporal_store(v[k], reinterpret_cast<nt4*>(base + k * step));
}

}  // namespace beam

// Room for at least B * K * spans_of() spans, in numbers that do not fall as any
// argument grows: a workspace sized for the largest call serves the smaller ones.
size_t beam_select_ws_bytes(int B, int K, int V, int S) {
    const int64_t rows = static_cast<int64_t>(B) * K;
    const int64_t per_row = std::min<int64_t>(std::max<int64_t>((static_cast<int64_t>(V) + 1023) / 1024, 4), beam::kMaxSpans);
    const int64_t slots = std::min(rows * per_row, std::max(4 * rows, 4096 + rows));
    return static_cast<size_t>(slots) * (sizeof(beam::Part) + sizeof(uint2) * static_cast<size_t>(S));
}

hipError_t launch_beam_select(const BeamGeo& g, const void* logits, const float* scores, const uint8_t* finished,
                              int eos, float* out_scores, int32_t* parent, int32_t* token, void* ws, hipStream_t s) {
    const int spans = beam::spans_of(g.B, g.K, g.V, g.S);
    const int64_t rows = static_cast<int64_t>(g.B) * g.K;
    beam::Part* sums = static_cast<beam::Part*>(ws);
    uint2* keys = reinterpret_cast<uint2*>(sums + rows * spans);
    const dim3 grid(static_cast<unsigned>(rows * (spans / 4))), block(256);
    if (g.bf16)
        hipLaunchKernelGGL(beam::beam_scan_kernel<uint16_t>, grid, block, 0, s, static_cast<const uint16_t*>(logits),
                           scores, finished, g.pitch, g.V, g.S, spans, sums, keys);
    else
        hipLaunchKernelGGL(beam::beam_scan_kernel<float>, grid, block, 0, s, static_cast<const float*>(logits),
                           scores, finished, g.pitch, g.V, g.S, spans, sums, keys);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const size_t lds = static_cast<size_t>(g.K) * spans * g.S * (sizeof(uint64_t) + sizeof(uint32_t) + sizeof(int));
    const int entries = g.K * spans * g.S;
    const auto join = entries <= 1024   ? beam::beam_join_kernel<1>
                      : entries <= 2048 ? beam::beam_join_kernel<2>
                                        : beam::beam_join_kernel<beam::kMaxEntries / (64 * beam::kJoinWaves)>;
    if (lds > 32768) {   // asked for well before static and dynamic part pass the 64 KB that need no asking
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(join), hipFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(lds));
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(join, dim3(static_cast<unsigned>(g.B)), dim3(64 * beam::kJoinWaves), lds, s,
                       sums, keys, scores, finished, eos, g.K, g.V, g.S, spans, out_scores, parent, token);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(int groups, int K, int64_t state_bytes, int64_t tail_bytes, void* state, void* tail,
                               const int32_t* parent, int32_t* status, hipStream_t s) {
    const int64_t su = state_bytes / 16, tu = tail_bytes / 16;
    const int wgs = static_cast<int>((su + tu + 255) / 256);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(groups) * wgs)), block(256);
    float *S = static_cast<float*>(state), *T = static_cast<float*>(tail);
    if (K <= 4)
        hipLaunchKernelGGL(beam::beam_reorder_kernel<4>, grid, block, 0, s, S, T, su, tu, K, parent, status, wgs);
    else if (K <= 8)
        hipLaunchKernelGGL(beam::beam_reorder_kernel<8>, grid, block, 0, s, S, T, su, tu, K, parent, status, wgs);
    else if (K <= 16)
        hipLaunchKernelGGL(beam::beam_reorder_kernel<16>, grid, block, 0, s, S, T, su, tu, K, parent, status, wgs);
    else
        hipLaunchKernelGGL(beam::beam_reorder_kernel<32>, grid, block, 0, s, S, T, su, tu, K, parent, status, wgs);
    return hipGetLastError();
}

}  // namespace gdn
