// gdn_beam.hip -- beam search over recurrent states: the selection over beams
// and vocabulary, and the move of the beams' states.
//
// Selection.  Candidate (k, v) of a sequence has the value
//   score_k + (l_kv - m_k) - log sum_v exp(l_kv - m_k),   m_k = max_v l_kv
// and the S best of the K*V are wanted, ties to the lowest k*V + v.  Within a
// beam the order is the order of its logits, so one pass over the logits keeps
// the running maximum, the sum of exponentials and the S best (logit, index)
// pairs of each span of a row; a second, small launch joins the spans.
//   scan  one wave per span of a row.  The wave's S best are a sorted list, one
//         entry per lane; a vector of logits is looked at closer only when its
//         largest reaches the list's S-th, which after the first few hundred
//         logits is rare.  Nothing but registers is used.
//   join  one workgroup per sequence: each beam's sum over the spans in fp64,
//         then the S best of the spans' lists by their fp64 value.
// Keys (ordered logit bits, complement of the index) are unique, so the result
// does not depend on the order in which spans or waves finish.
#include "gdn.h"
#include "gdn_core.hpp"
#include "gdn_launch.hpp"

namespace gdn {
namespace beam {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSpans = 64;

// A masked or broken logit (NaN) counts as -inf; +inf counts as the largest
// finite value, so that a row keeps a finite maximum; -0 becomes +0.
__device__ __forceinline__ float clean(float v) {
    v = v == v ? v : -__builtin_inff();
    return fminf(v, __FLT_MAX__) + 0.0f;
}
// Order-preserving map of a clean float to an unsigned integer; 0 is below all.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ uint32_t from_lane_below(uint32_t v) { return __shfl_up(v, 1); }

// The S best keys of a wave, best first, one per lane.
struct Best {
    uint32_t hi = 0, lo = 0;   // this lane's entry; 0, 0 is none
    uint32_t th = 0, tl = 0;   // entry S - 1, in every lane

    __device__ void insert(uint32_t h, uint32_t l, int lane, int S) {   // h, l uniform
        const bool better = hi > h || (hi == h && lo > l);
        const int at = __popcll(__ballot(better));
        const uint32_t uh = from_lane_below(hi), ul = from_lane_below(lo);
        if (lane == at) {
            hi = h;
            lo = l;
        } else if (lane > at) {
            hi = uh;
            lo = ul;
        }
        th = lane_of(hi, S - 1);
        tl = lane_of(lo, S - 1);
    }
    // One candidate in each lane of `want`.
    __device__ void offer(uint32_t h, uint32_t l, bool want, int lane, int S) {
        uint64_t todo = __ballot(want && (h > th || (h == th && l > tl)));
        while (todo) {
            const int from = __builtin_ctzll(todo);
            todo &= todo - 1;
            const uint32_t ch = lane_of(h, from), cl = lane_of(l, from);
            if (ch > th || (ch == th && cl > tl))
                insert(ch, cl, lane, S);
        }
    }
};

template <typename Act>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int E = 8;
    __device__ static void load(const uint16_t* p, float v[8]) {
        typedef uint32_t u4 __attribute__((ext_vector_type(4)));
        const u4 r = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(r[j] << 16);
            v[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
        }
    }
};
template <>
struct Vec<float> {
    static constexpr int E = 4;
    __device__ static void load(const float* p, float v[4]) {
        const nt4 r = __builtin_nontemporal_load(reinterpret_cast<const nt4*>(p));
        v[0] = r.x;
        v[1] = r.y;
        v[2] = r.z;
        v[3] = r.w;
    }
};

// A span's maximum and its sum of exponentials.  The sum is kept in fp64: what
// it loses shifts every candidate of the beam against the other beams'.
struct alignas(16) Part {
    double s;
    float m, unused;
};

// Running maximum and sum of exponentials of one lane.
struct Sum {
    float m = -__builtin_inff(), s = 0.0f;
    template <int E>
    __device__ float add(const float (&v)[E]) {
        float top = v[0];
#pragma unroll
        for (int e = 1; e < E; ++e)
            top = fmaxf(top, v[e]);
        if (top > m) {
            s *= __builtin_amdgcn_exp2f((m - top) * kLog2e);   // m = -inf: s is 0 and stays 0
            m = top;
        }
        const float ref = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < E; ++e)
            s += __builtin_amdgcn_exp2f((v[e] - ref) * kLog2e);
        return top;
    }
};

template <typename Act>
__global__ __launch_bounds__(256) void beam_scan_kernel(const Act* __restrict__ logits, int64_t pitch, int V, int S,
                                                        int spans, Part* __restrict__ sums,
                                                        uint2* __restrict__ keys) {
    constexpr int E = Vec<Act>::E;
    const int lane = threadIdx.x & (kWave - 1);
    const int wgs = spans / 4;
    const int64_t row = blockIdx.x / wgs;
    const int span = (blockIdx.x % wgs) * 4 + threadIdx.x / kWave;
    const Act* p = logits + row * pitch;
    // logits before the first 16-byte boundary of the row, and whole vectors after it
    int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / static_cast<int>(sizeof(Act));
    head = head < V ? head : V;
    const int nvec = (V - head) / E;
    const int per = (nvec + spans - 1) / spans;
    const int v0 = span * per < nvec ? span * per : nvec;
    const int v1 = v0 + per < nvec ? v0 + per : nvec;

    Best best;
    Sum sum;
    // the row's ends: fewer than E logits before the vectors and fewer than E after
    if (span == 0) {
        const int tail0 = head + nvec * E;
        const int i = lane < head ? lane : tail0 + lane - head;
        const bool in = i < V;
        float v[1] = {in ? clean(widen(p[i])) : -__builtin_inff()};
        sum.add(v);
        best.offer(ordered(v[0]), ~static_cast<uint32_t>(i), in, lane, S);
    }
    for (int j = v0; j < v1; j += kWave) {
        const bool in = j + lane < v1;
        const int i0 = head + (in ? j + lane : v0) * E;
        float v[E];
        Vec<Act>::load(p + i0, v);
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] = in ? clean(v[e]) : -__builtin_inff();
        const float top = sum.add(v);
        if (__ballot(in && ordered(top) >= best.th)) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                best.offer(ordered(v[e]), ~static_cast<uint32_t>(i0 + e), in, lane, S);
        }
    }
    // the wave's maximum and sum
    float m = sum.m;
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1)
        m = fmaxf(m, __shfl_xor(m, k));
    const float ref = m == -__builtin_inff() ? 0.0f : m;
    double s = static_cast<double>(sum.s) * static_cast<double>(__builtin_amdgcn_exp2f((sum.m - ref) * kLog2e));
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1)
        s += __shfl_xor(s, k);
    const int64_t slot = row * spans + span;
    if (lane == 0)
        sums[slot] = Part{s, m, 0.0f};
    if (lane < S)
        keys[slot * S + lane] = make_uint2(best.hi, best.lo);
}

// fp64 counterpart of the ordered map.
__device__ __forceinline__ uint64_t ordered64(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double unordered64(uint64_t o) {
    return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}
__device__ __forceinline__ uint64_t lane_of64(uint64_t v, int lane) {
    return static_cast<uint64_t>(lane_of(static_cast<uint32_t>(v >> 32), lane)) << 32 |
           lane_of(static_cast<uint32_t>(v), lane);
}

// The same sorted list by fp64 value, then lowest flat index (kept complemented).
struct Best64 {
    uint64_t val = 0, tv = 0;
    uint32_t idx = 0, ti = 0;
    __device__ void offer(uint64_t v, uint32_t i, bool want, int lane, int S) {
        uint64_t todo = __ballot(want && (v > tv || (v == tv && i > ti)));
        while (todo) {
            const int from = __builtin_ctzll(todo);
            todo &= todo - 1;
            const uint64_t cv = lane_of64(v, from);
            const uint32_t ci = lane_of(i, from);
            if (!(cv > tv || (cv == tv && ci > ti)))
                continue;
            const int at = __popcll(__ballot(val > cv || (val == cv && idx > ci)));
            const uint64_t uv = static_cast<uint64_t>(from_lane_below(static_cast<uint32_t>(val >> 32))) << 32 |
                                from_lane_below(static_cast<uint32_t>(val));
            const uint32_t ui = from_lane_below(idx);
            if (lane == at) {
                val = cv;
                idx = ci;
            } else if (lane > at) {
                val = uv;
                idx = ui;
            }
            tv = lane_of64(val, S - 1);
            ti = lane_of(idx, S - 1);
        }
    }
};

__global__ __launch_bounds__(256) void beam_join_kernel(const Part* __restrict__ sums,
                                                        const uint2* __restrict__ keys,
                                                        const float* __restrict__ scores,
                                                        const uint8_t* __restrict__ finished, int eos, int K, int V,
                                                        int S, int spans, float* __restrict__ out_scores,
                                                        int32_t* __restrict__ parent, int32_t* __restrict__ token) {
    __shared__ uint64_t lv[3 * kWave];
    __shared__ uint32_t li[3 * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int64_t seq = blockIdx.x;
    const uint64_t none = ordered64(-__builtin_inf());
    Best64 best;
    for (int k = wave; k < K; k += 4) {
        const int64_t row = seq * K + k;
        const float sc = clean(scores[row]);
        const uint32_t flat0 = static_cast<uint32_t>(k) * static_cast<uint32_t>(V);
        const bool fin = finished && finished[row];
        // the beam's maximum and sum over its spans (at most one per lane)
        const Part part = lane < spans ? sums[row * spans + lane] : Part{0.0, -__builtin_inff(), 0.0f};
        float m = part.m;
#pragma unroll
        for (int j = 32; j >= 1; j >>= 1)
            m = fmaxf(m, __shfl_xor(m, j));
        const bool dead = sc == -__builtin_inff() || (!fin && m == -__builtin_inff());
        if (dead || fin) {
            // at most one live candidate (the end token at the beam's own score); all others are -inf
            const int t = fin && !dead ? (lane == 0 ? eos : lane - 1 < eos ? lane - 1 : lane) : lane;
            const uint64_t v = fin && !dead && lane == 0 ? ordered64(static_cast<double>(sc)) : none;
            best.offer(v, ~(flat0 + static_cast<uint32_t>(t)), t < V, lane, S);
            continue;
        }
        double s = part.m == -__builtin_inff() ? 0.0 : part.s * exp(static_cast<double>(part.m) - m);
#pragma unroll
        for (int j = 32; j >= 1; j >>= 1)
            s += __shfl_xor(s, j);
        const double logs = log(s);
        const int n = spans * S;
        for (int e0 = 0; e0 < n; e0 += kWave) {
            const int e = e0 + lane;
            const uint2 q = e < n ? keys[row * n + e] : make_uint2(0, 0);
            const double l = static_cast<double>(unordered(q.x));
            const double v = static_cast<double>(sc) + ((l - m) - logs);
            best.offer(ordered64(v + 0.0), ~(flat0 + ~q.y), q.x != 0, lane, S);
        }
    }
    if (wave > 0) {
        lv[(wave - 1) * kWave + lane] = best.val;
        li[(wave - 1) * kWave + lane] = best.idx;
    }
    __syncthreads();
    if (wave == 0) {
        for (int w = 0; w < 3; ++w)
            best.offer(lv[w * kWave + lane], li[w * kWave + lane], lv[w * kWave + lane] != 0, lane, S);
        if (lane < S) {
            const uint32_t flat = ~best.idx;
            out_scores[seq * S + lane] = static_cast<float>(unordered64(best.val));
            parent[seq * S + lane] = static_cast<int32_t>(flat / static_cast<uint32_t>(V));
            token[seq * S + lane] = static_cast<int32_t>(flat % static_cast<uint32_t>(V));
        }
    }
}

// Spans per row: enough waves to fill the chip (8,192) over all rows, spans of
// at least 1,024 logits, at most one span per lane of the joining wave.
static int spans_of(int B, int K, int V) {
    const int64_t rows = static_cast<int64_t>(B) * K;
    int64_t n = (8192 + rows - 1) / rows;
    const int64_t most = (static_cast<int64_t>(V) + 1023) / 1024;
    n = n < most ? n : most;
    n = n < kMaxSpans ? n : kMaxSpans;
    return static_cast<int>((n + 3) / 4 * 4);
}

// Reorder.  A thread owns one 16-byte unit of a sequence's state (or tail) in
// every slot of its group: it loads, for each slot that takes another's state,
// the unit from that slot's parent, and stores only after its last load.  No
// other thread touches those units, so the move is in place without a second
// copy of the states, and slots that keep their own state cost nothing.  Bound
// by HBM: the sources that move are read, the slots that move are written.
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
    float4 v[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (from[k] != k)
            v[k] = *reinterpret_cast<const float4*>(base + from[k] * step);
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (from[k] != k)
            *reinterpret_cast<float4*>(base + k * step) = v[k];
}

}  // namespace beam

size_t beam_select_ws_bytes(int B, int K, int V, int S) {
    const size_t slots = static_cast<size_t>(B) * K * beam::spans_of(B, K, V);
    return slots * (sizeof(beam::Part) + sizeof(uint2) * static_cast<size_t>(S));
}

hipError_t launch_beam_select(const BeamGeo& g, const void* logits, const float* scores, const uint8_t* finished,
                              int eos, float* out_scores, int32_t* parent, int32_t* token, void* ws, hipStream_t s) {
    const int spans = beam::spans_of(g.B, g.K, g.V);
    const int64_t rows = static_cast<int64_t>(g.B) * g.K;
    beam::Part* sums = static_cast<beam::Part*>(ws);
    uint2* keys = reinterpret_cast<uint2*>(sums + rows * spans);
    const dim3 grid(static_cast<unsigned>(rows * (spans / 4))), block(256);
    if (g.bf16)
        hipLaunchKernelGGL(beam::beam_scan_kernel<uint16_t>, grid, block, 0, s, static_cast<const uint16_t*>(logits),
                           g.pitch, g.V, g.S, spans, sums, keys);
    else
        hipLaunchKernelGGL(beam::beam_scan_kernel<float>, grid, block, 0, s, static_cast<const float*>(logits),
                           g.pitch, g.V, g.S, spans, sums, keys);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(beam::beam_join_kernel, dim3(static_cast<unsigned>(g.B)), block, 0, s, sums, keys, scores,
                       finished, eos, g.K, g.V, g.S, spans, out_scores, parent, token);
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
