// gdn_norm.hip -- the norms on either side of a block: the residual sum with
// the norm before the next block, and the norm of a mixer's output with its
// gate; both with their gradients.
//
// A row (of the residual stream, or of one head) is held in the registers of a
// team of lanes: part of a wave, or a workgroup, so that every value is read
// once and written once.  All of it is fp32 but for what is stored.
//
// HBM sets the time of long calls, the launch that of a few rows (64 rows of 5,120:
// 3.5 us; 64 x 48 heads of 128: 2.8 us).  Measured, where a copy of 1 GiB runs at
// 5.2 TB/s: 32,768 rows of 5,120 with an fp32 stream, scale and w_post 362-368 us, 5.5
// TB/s; 8,192 x 48 heads of 128 from fp32 with gate 70 us forward, 120 us backward,
// 5.8 TB/s.  Non-temporal loads and stores are worth 383 -> 367 and 212 -> 202 us.
#include "gdn.h"
#include "gdn_lru.hpp"

namespace gdn {
namespace norm {

using lru::silu;
using lru::silu_slope;

constexpr int kMaxSums = 3;     // weight gradients of one call

// U consecutive values of a row: read once and written once, past what the caches
// hold for reuse.
template <typename T, int U>
struct Unit;
template <int U>
struct Unit<uint16_t, U> {
    static constexpr int WORDS = U / 2, VALUES = U;
    typedef uint32_t raw __attribute__((ext_vector_type(WORDS)));
    __device__ static raw load(const uint16_t* p) { return __builtin_nontemporal_load(reinterpret_cast<const raw*>(p)); }
    __device__ static void to_float(raw v, float (&f)[U]) {
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            f[2 * k] = __uint_as_float(v[k] << 16);
            f[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
        }
    }
    __device__ static void store(uint16_t* p, const float (&f)[U]) {
        raw v;
#pragma unroll
        for (int k = 0; k < WORDS; k += 2) {
            const float four[4] = {f[2 * k], f[2 * k + 1], f[2 * k + 2], f[2 * k + 3]};
            const uint2 w = lru::pack(four, uint16_t());
            v[k] = w.x;
            v[k + 1] = w.y;
        }
        __builtin_nontemporal_store(v, reinterpret_cast<raw*>(p));
    }
};
template <>
struct Unit<float, 4> {
    static constexpr int VALUES = 4;
    typedef float raw __attribute__((ext_vector_type(4)));
    __device__ static raw load(const float* p) { return __builtin_nontemporal_load(reinterpret_cast<const raw*>(p)); }
    __device__ static void to_float(raw v, float (&f)[4]) { f[0] = v[0], f[1] = v[1], f[2] = v[2], f[3] = v[3]; }
    __device__ static void store(float* p, const float (&f)[4]) {
        __builtin_nontemporal_store(raw{f[0], f[1], f[2], f[3]}, reinterpret_cast<raw*>(p));
    }
};
// Element c of a row.  The row is the same for a whole wave where a workgroup shares
// it, and an offset of 32 bits then needs no address of its own in registers.
template <typename T>
__device__ __forceinline__ T* spot(T* row, uint32_t c) {
    return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(row) + c * static_cast<uint32_t>(sizeof(T)));
}

// Keeps values as they were read: what is widened behind this is widened again, and not
// held in twice the registers since before it.
template <typename RAW>
__device__ __forceinline__ void hold_raw(RAW& v) {
#pragma unroll
    for (unsigned k = 0; k < sizeof(RAW) / 4; ++k) {
        auto word = v[k];
        asm volatile("" : "+v"(word));
        v[k] = word;
    }
}

// A column that the compiler takes for a new one: weights that do not fit the registers
// are read where they are used, and not all ahead of the loop over the rows.
__device__ __forceinline__ uint32_t anew(uint32_t c) {
    asm volatile("" : "+v"(c));
    return c;
}

// Weights are read by every row.
template <int U>
__device__ __forceinline__ void load_weight(const float* p, float (&f)[U]) {
#pragma unroll
    for (int k = 0; k < U; k += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + k);
        f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
    }
}

template <typename A, typename B>
constexpr int unit_of() { return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4; }

// A team: LPR lanes of a wave (LPR <= 64), or a whole workgroup (LPR == 0).
template <int LPR>
struct Team {
    int index, slot, size, teams, flip = 0;
    float* mem;   // 2 x 48 floats, workgroup teams only
    __device__ explicit Team(float* m)
        : index(LPR ? threadIdx.x % (LPR ? LPR : 1) : threadIdx.x), slot(LPR ? threadIdx.x / (LPR ? LPR : 1) : 0),
          size(LPR ? LPR : blockDim.x), teams(LPR ? blockDim.x / (LPR ? LPR : 1) : 1), mem(m) {}
    // Sums of K values over the team, in a fixed order, in all of its lanes.
    template <int K>
    __device__ void sum(float (&v)[K]) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (LPR == 32) {
                v[k] = group_sum<16>(v[k]);
                v[k] += __shfl_xor(v[k], 16);
            } else {
                v[k] = group_sum<LPR ? LPR : 64>(v[k]);
            }
        }
        if constexpr (LPR == 0) {
            float* m = mem + flip;
            flip ^= 48;
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    m[k * 16 + (threadIdx.x >> 6)] = v[k];
            __syncthreads();
            const int waves = blockDim.x >> 6;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float s = 0.0f;
                for (int w = 0; w < waves; ++w)
                    s += m[k * 16 + w];
                v[k] = s;
            }
        }
    }
};

// What a kernel needs of a row's length n.
struct Mean {
    float inv_n, eps;
    float unit, inv_square;   // a power of two of at most n^-1/2; 1 / (n unit^2)
    Mean(int n, float e) : inv_n(1.0f / n), eps(e), unit(1.0f), inv_square(inv_n) {
        for (int covered = 1; covered < n; covered *= 4) {
            unit *= 0.5f;
            inv_square *= 4.0f;
        }
    }
};

// 1 / sqrt(mean square + eps) from the sum of a row's squares, in all lanes of its team.
// The sum may be beyond fp32 where the mean is not (16,384 values of 2e17: 6.6e38 and
// 4e34); such a row's squares are summed again, as those of its values times `unit`,
// which stay below their mean.  values(f) calls f with each of the lane's values.
template <int LPR, typename F>
__device__ __forceinline__ float inv_rms(Team<LPR>& team, const Mean& mean, float squares, F values) {
    float inv = mean.inv_n;
    if (__builtin_expect(squares == __builtin_inff(), 0)) {
        float again[1] = {0.0f};
        values([&](float v) {
            const float u = v * mean.unit;
            again[0] = __builtin_fmaf(u, u, again[0]);
        });
        team.sum(again);
        squares = again[0];
        inv = mean.inv_square;
    }
    return __builtin_amdgcn_rsqf(__builtin_fmaf(squares, inv, mean.eps));
}

// A lane's values of a row, as numbers and as they were read.
template <int NV, int U, typename F>
__device__ __forceinline__ void each(const bool (&on)[NV], const float (&v)[NV][U], F f) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (on[j])
#pragma unroll
            for (int k = 0; k < U; ++k)
                f(v[j][k]);
}
template <typename UNIT, int NV, typename F>
__device__ __forceinline__ void each_raw(const bool (&on)[NV], const typename UNIT::raw (&raw)[NV], F f) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float v[UNIT::VALUES];
        UNIT::to_float(raw[j], v);
        if (on[j])
#pragma unroll
            for (int k = 0; k < UNIT::VALUES; ++k)
                f(v[k]);
    }
}

// ------------------------------------------------------------ residual and norm

template <typename Act, typename Res, int U, int LPR, int NV, bool POST>
__global__ __launch_bounds__(LPR ? 256 : 1024) void residual_norm_kernel(
    const Res* residual, const Act* __restrict__ delta, const float* __restrict__ scale,
    const float* __restrict__ post, const float* __restrict__ w, Res* out, Act* __restrict__ y, int64_t rows, int W,
    Mean mean) {
    __shared__ float mem[96];
    Team<LPR> team(mem);
    using RU = Unit<Res, U>;
    using AU = Unit<Act, U>;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * team.teams + team.slot; row < rows;
         row += static_cast<int64_t>(gridDim.x) * team.teams) {
        const int64_t base = row * W;
        float s[NV][U], d[NV][U], sq[1];
        bool on[NV];
        uint32_t c[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int u = (team.index + j * team.size) * U;
            on[j] = u < W;
            c[j] = on[j] ? u : 0;
            if (delta)
                AU::to_float(AU::load(spot(delta + base, c[j])), d[j]);
            RU::to_float(RU::load(spot(residual + base, c[j])), s[j]);
        }
        if (delta) {
            float p = 1.0f;
            if constexpr (POST) {
                sq[0] = 0.0f;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int k = 0; k < U; ++k)
                        sq[0] = on[j] ? __builtin_fmaf(d[j][k], d[j][k], sq[0]) : sq[0];
                team.sum(sq);
                p = inv_rms(team, mean, sq[0], [&](auto f) { each(on, d, f); });
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float ws[U], wp[U];
                if (scale)
                    load_weight<U>(spot(scale, c[j]), ws);
                if constexpr (POST)
                    load_weight<U>(spot(post, c[j]), wp);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const float n = POST ? d[j][k] * p * wp[k] : d[j][k];
                    s[j][k] = scale ? __builtin_fmaf(ws[k], n, s[j][k]) : s[j][k] + n;
                    if constexpr (sizeof(Res) == 2)   // y is the norm of the stream as it is stored
                        s[j][k] = static_cast<float>(static_cast<__bf16>(s[j][k]));
                }
                if (on[j])
                    RU::store(spot(out + base, c[j]), s[j]);
            }
        }
        sq[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < U; ++k)
                sq[0] = on[j] ? __builtin_fmaf(s[j][k], s[j][k], sq[0]) : sq[0];
        team.sum(sq);
        const float q = inv_rms(team, mean, sq[0], [&](auto f) { each(on, s, f); });
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float ww[U];
            load_weight<U>(spot(w, c[j]), ww);
#pragma unroll
            for (int k = 0; k < U; ++k)
                ww[k] *= s[j][k] * q;
            if (on[j])
                AU::store(spot(y + base, c[j]), ww);
        }
    }
}

// Adds the teams' sums of one workgroup in a fixed order and writes them as row
// blockIdx.x of parts; sums is what each thread gathered for its columns.
template <int LPR, int U, int NV>
__device__ __forceinline__ void write_part(const Team<LPR>& team, float (&sums)[NV][U], int W, float* lds,
                                           float* __restrict__ part) {
    if constexpr (LPR == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (team.index + j * team.size) * U;
            if (c < W)
#pragma unroll
                for (int k = 0; k < U; ++k)
                    part[c + k] = sums[j][k];
        }
    } else {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < U; ++k)
                lds[(team.slot * NV + j) * LPR * U + team.index * U + k] = sums[j][k];
        __syncthreads();
        for (int c = threadIdx.x; c < W; c += blockDim.x) {
            const int j = c / (LPR * U), in = c % (LPR * U);
            float s = 0.0f;
            for (int t = 0; t < team.teams; ++t)
                s += lds[(t * NV + j) * LPR * U + in];
            part[c] = s;
        }
    }
}

// A workgroup walks rows, so that the weights' gradients stay in its registers (and
// the weights with them).  Two sums to wait for per row (three values, then with
// `post` one), the next row asked for before them: 8,192 rows of 4,096 bf16 from 195
// to 98 us (403 MB, and 25 MB of parts), with the sums one by one and no row ahead.
template <typename Act, typename Res, int U, int LPR, int NV, bool POST>
__global__ __launch_bounds__(LPR ? 256 : 1024) void residual_norm_backward_kernel(
    const Res* __restrict__ stream, const Act* __restrict__ delta, const float* __restrict__ scale,
    const float* __restrict__ post, const float* __restrict__ w, const Act* __restrict__ dy, const Res* ds,
    Res* dres, Act* __restrict__ ddelta, float* __restrict__ parts, int64_t rows, int W, Mean mean) {
    __shared__ float mem[96];
    __shared__ float lds[LPR ? 256 * NV * U : 1];
    Team<LPR> team(mem);
    using RU = Unit<Res, U>;
    using AU = Unit<Act, U>;
    // of wide rows neither the weights nor the sums for scale and w_post fit the registers,
    // of the widest not the next row either; the sums then lie in LDS, each lane's own
    // (training step of 3,161 rows of 8,680 in bf16 200 us, 338 with them in registers;
    // 8,192 of 5,120 in fp32 336 and 373)
    constexpr bool KEEP = NV == 1, AHEAD = NV <= 2, APART = NV > 1;
    __shared__ float4 apart[2][APART ? NV * 1024 : 1];
    float sw[NV][U] = {}, ss[NV][U] = {}, sp[NV][U] = {}, ww[NV][U], ws[NV][U], wp[NV][U];
    bool on[NV];
    uint32_t c[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int u = (team.index + j * team.size) * U;
        on[j] = u < W;
        c[j] = on[j] ? u : 0;
    }
    if constexpr (APART)
#pragma unroll
        for (int j = 0; j < NV; ++j)
            apart[0][team.index + j * team.size] = apart[1][team.index + j * team.size] = make_float4(0, 0, 0, 0);
    auto weigh_norm = [&](int j) { load_weight<U>(spot(w, KEEP ? c[j] : anew(c[j])), ww[j]); };
    auto weigh_delta = [&](int j) {
        const uint32_t at = KEEP ? c[j] : anew(c[j]);
        if (scale)
            load_weight<U>(spot(scale, at), ws[j]);
        else
#pragma unroll
            for (int k = 0; k < U; ++k)
                ws[j][k] = 1.0f;
        if constexpr (POST)
            load_weight<U>(spot(post, at), wp[j]);
    };
    if constexpr (KEEP) {
        weigh_norm(0);
        weigh_delta(0);
    }
    typename RU::raw rs[NV], rt[NV] = {};
    typename AU::raw rg[NV], rd[NV] = {};
    auto ask = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            rs[j] = RU::load(spot(stream + row * W, c[j]));
            rg[j] = AU::load(spot(dy + row * W, c[j]));
            if (delta)
                rd[j] = AU::load(spot(delta + row * W, c[j]));
            if (ds)
                rt[j] = RU::load(spot(ds + row * W, c[j]));
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * team.teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * team.teams + team.slot;
    if (AHEAD && row < rows)
        ask(row);
    for (; row < rows; row += step) {
        const int64_t base = row * W;
        float sums[POST ? 3 : 2] = {};
        typename RU::raw cs[NV], ct[NV];
        typename AU::raw cg[NV], cd[NV];
        if constexpr (!AHEAD)
            ask(row);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            cs[j] = rs[j], cg[j] = rg[j], cd[j] = rd[j], ct[j] = rt[j];
        if (AHEAD && row + step < rows)
            ask(row + step);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (!KEEP)
                weigh_norm(j);
            float s[U], g[U], d[U];
            RU::to_float(cs[j], s);
            AU::to_float(cg[j], g);
            AU::to_float(cd[j], d);
            if (on[j])
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    sums[0] = __builtin_fmaf(s[k], s[k], sums[0]);
                    sums[1] = __builtin_fmaf(g[k] * ww[j][k], s[k], sums[1]);
                    if constexpr (POST)
                        sums[2] = __builtin_fmaf(d[k], d[k], sums[2]);
                }
            if constexpr (!KEEP) {
                hold_raw(cs[j]);
                hold_raw(cg[j]);
                hold_raw(cd[j]);
            }
        }
        team.sum(sums);
        const float q = inv_rms(team, mean, sums[0], [&](auto f) { each_raw<RU>(on, cs, f); });
        const float back = q * q * (sums[1] * mean.inv_n);
        const float p = POST ? inv_rms(team, mean, sums[POST ? 2 : 0], [&](auto f) { each_raw<AU>(on, cd, f); }) : 1.0f;
        float t[NV][U], dot[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (!KEEP) {
                weigh_norm(j);
                weigh_delta(j);
            }
            float s[U], g[U], d[U];
            RU::to_float(cs[j], s);
            AU::to_float(cg[j], g);
            AU::to_float(cd[j], d);
            RU::to_float(ct[j], t[j]);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                sw[j][k] = __builtin_fmaf(g[k], s[k] * q, sw[j][k]);
                t[j][k] = __builtin_fmaf(q, g[k] * ww[j][k] - s[k] * back, t[j][k]);
            }
            if (on[j])
                RU::store(spot(dres + base, c[j]), t[j]);
            float as[U], ap[U];   // the sums' values of this unit
            auto fetch = [&](int which, float (&own)[U], float (&v)[U]) {
                if constexpr (APART)
                    load_weight<U>(reinterpret_cast<const float*>(&apart[which][team.index + j * team.size]), v);
                else
#pragma unroll
                    for (int k = 0; k < U; ++k)
                        v[k] = own[k];
            };
            auto keep = [&](int which, float (&own)[U], const float (&v)[U]) {
                if constexpr (APART)
                    apart[which][team.index + j * team.size] = make_float4(v[0], v[1], v[2], v[3]);
                else
#pragma unroll
                    for (int k = 0; k < U; ++k)
                        own[k] = v[k];
            };
            fetch(0, ss[j], as);
            if constexpr (POST)
                fetch(1, sp[j], ap);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const float dn = d[k] * p;
                as[k] = __builtin_fmaf(t[j][k], POST ? dn * wp[j][k] : dn, as[k]);
                t[j][k] *= ws[j][k];
                if constexpr (POST) {
                    ap[k] = __builtin_fmaf(t[j][k], dn, ap[k]);
                    t[j][k] *= wp[j][k];
                    if (on[j])
                        dot[0] = __builtin_fmaf(t[j][k], d[k], dot[0]);
                }
            }
            keep(0, ss[j], as);
            if constexpr (POST)
                keep(1, sp[j], ap);
            if constexpr (!KEEP)
                hold_raw(cd[j]);
        }
        if (!delta)
            continue;
        if constexpr (POST) {
            team.sum(dot);
            const float back2 = p * p * (dot[0] * mean.inv_n);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float d[U];
                    AU::to_float(cd[j], d);
#pragma unroll
                for (int k = 0; k < U; ++k)
                    t[j][k] = p * (t[j][k] - d[k] * back2);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (on[j])
                AU::store(spot(ddelta + base, c[j]), t[j]);
    }
    const int64_t plane = static_cast<int64_t>(gridDim.x) * W;
    float* part = parts + static_cast<int64_t>(blockIdx.x) * W;
    if constexpr (APART)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            load_weight<U>(reinterpret_cast<const float*>(&apart[0][team.index + j * team.size]), ss[j]);
            load_weight<U>(reinterpret_cast<const float*>(&apart[1][team.index + j * team.size]), sp[j]);
        }
    write_part<LPR, U, NV>(team, sw, W, lds, part);
    if (delta && scale)
        write_part<LPR, U, NV>(team, ss, W, lds, part + plane);
    if constexpr (POST)
        write_part<LPR, U, NV>(team, sp, W, lds, part + 2 * plane);
}

struct Sums {
    float* out[kMaxSums];
};

// Column sums of the workgroups' parts, in a fixed order, 64 columns at a time.
// blockIdx.y: which.
__global__ __launch_bounds__(1024) void part_sum_kernel(const float* __restrict__ parts, Sums sums, int rows, int W) {
    __shared__ float mem[16][64];
    float* out = sums.out[blockIdx.y];
    if (!out)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * 64; first < W; first += static_cast<int64_t>(gridDim.x) * 64) {
        const int64_t c = first + lane;
        const float* p = parts + static_cast<int64_t>(blockIdx.y) * rows * W + c;
        float s = 0.0f;
        if (c < W)
#pragma unroll 8
            for (int row = wave; row < rows; row += 16)
                s += p[static_cast<int64_t>(row) * W];
        mem[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && c < W) {
            float t = 0.0f;
            for (int w = 0; w < 16; ++w)
                t += mem[w][lane];
            out[c] = t;
        }
        __syncthreads();
    }
}
// Workgroups of 1,024 for so many columns; a launch counts 2^32 threads, and the weights
// of 65,536 heads of 4,096 would be as many.
constexpr int64_t kSumBlocks = 1 << 20;
inline unsigned sum_blocks(int64_t columns) {
    const int64_t need = (columns + 63) / 64;
    return static_cast<unsigned>(need < kSumBlocks ? need : kSumBlocks);
}

// ------------------------------------------------------------ norm and gate

template <typename O, typename Act, int U, int LPR, int NV, bool FIRST>
__global__ __launch_bounds__(LPR ? 256 : 1024) void gated_norm_kernel(
    const O* __restrict__ o, const Act* __restrict__ z, const float* __restrict__ w, Act* __restrict__ y,
    int64_t items, int H, int D, int64_t z_pitch, int w_step, Mean mean) {
    __shared__ float mem[96];
    Team<LPR> team(mem);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * team.teams + team.slot; item < items;
         item += static_cast<int64_t>(gridDim.x) * team.teams) {
        const int64_t row = static_cast<uint32_t>(item) / static_cast<uint32_t>(H);   // fewer than 2^31 items
        const int h = static_cast<int>(item - row * H);
        float v[NV][U], gate[NV][U];
        bool on[NV];
        uint32_t c[NV];
        float sq[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int u = (team.index + j * team.size) * U;
            on[j] = u < D;
            c[j] = on[j] ? u : 0;
            Unit<O, U>::to_float(Unit<O, U>::load(spot(o + item * D, c[j])), v[j]);
            Unit<Act, U>::to_float(Unit<Act, U>::load(spot(z + row * z_pitch + static_cast<int64_t>(h) * D, c[j])), gate[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < U; ++k) {
                gate[j][k] = silu(gate[j][k]);
                if constexpr (FIRST)
                    v[j][k] *= gate[j][k];
                sq[0] = on[j] ? __builtin_fmaf(v[j][k], v[j][k], sq[0]) : sq[0];
            }
        // a head in part of a wave asks for its weights before it waits for the sum: 68.5 us against
        // 71.5 behind it; of wider rows they would only hold registers (8,192 of 5,120: 44.7 and 42.9)
        constexpr bool EARLY = LPR != 0;
        float ww[NV][U];
        auto weigh = [&](int j) { load_weight<U>(spot(w + static_cast<int64_t>(h) * w_step, c[j]), ww[j]); };
        if constexpr (EARLY)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                weigh(j);
        team.sum(sq);
        const float q = inv_rms(team, mean, sq[0], [&](auto f) { each(on, v, f); });
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (!EARLY)
                weigh(j);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                ww[j][k] *= v[j][k] * q;
                if constexpr (!FIRST)
                    ww[j][k] *= gate[j][k];
            }
            if (on[j])
                Unit<Act, U>::store(spot(y + item * D, c[j]), ww[j]);
        }
    }
}

// Team g keeps head g % H and walks every `step`-th row, so that its weight
// gradient stays in registers.  768 workgroups: 192 us for the training step of 8,192
// x 48 heads of 128 against 216-223 with 512 and 203 with 1,024.  One weight for all heads: parts [blocks][D], else
// [step][H][D].
template <typename O, typename Act, int U, int LPR, int NV, bool FIRST>
__global__ __launch_bounds__(LPR ? 256 : 1024) void gated_norm_backward_kernel(
    const O* __restrict__ o, const Act* __restrict__ z, const float* __restrict__ w, const Act* __restrict__ dy,
    O* __restrict__ dov, Act* __restrict__ dz, float* __restrict__ parts, int64_t rows, int H, int D, int64_t step,
    int64_t z_pitch, int64_t dz_pitch, int w_step, Mean mean) {
    __shared__ float mem[96];
    __shared__ float lds[LPR ? 256 * NV * U : 1];
    Team<LPR> team(mem);
    const int64_t id = static_cast<int64_t>(blockIdx.x) * team.teams + team.slot;
    const int h = static_cast<int>(id % H);
    const int64_t first = id / H;
    constexpr bool KEEP = NV == 1;   // of wider rows the gates are taken twice and the weights read again
    float sw[NV][U] = {}, ww[NV][U];
    bool on[NV];
    uint32_t c[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int u = (team.index + j * team.size) * U;
        on[j] = u < D;
        c[j] = on[j] ? u : 0;
    }
    auto weigh = [&](int j) {
        load_weight<U>(spot(w + static_cast<int64_t>(h) * w_step, KEEP ? c[j] : anew(c[j])), ww[j]);
    };
    if constexpr (KEEP)
        weigh(0);
    if (first < step)
        for (int64_t row = first; row < rows; row += step) {
            const int64_t base = (row * H + h) * D;
            typename Unit<O, U>::raw ro[NV];
            typename Unit<Act, U>::raw rz[NV], rg[NV];
            float gate[NV][U], slope[NV][U], sums[2] = {};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                ro[j] = Unit<O, U>::load(spot(o + base, c[j]));
                rz[j] = Unit<Act, U>::load(spot(z + row * z_pitch + static_cast<int64_t>(h) * D, c[j]));
                rg[j] = Unit<Act, U>::load(spot(dy + base, c[j]));
            }
            auto open = [&](int j) {
                float v[U];
                Unit<Act, U>::to_float(rz[j], v);
#pragma unroll
                for (int k = 0; k < U; ++k)
                    silu_slope(v[k], gate[j][k], slope[j][k]);
            };
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if constexpr (!KEEP)
                    weigh(j);
                open(j);
                float v[U], g[U];
                Unit<O, U>::to_float(ro[j], v);
                Unit<Act, U>::to_float(rg[j], g);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const float u = FIRST ? v[k] * gate[j][k] : v[k];
                    const float dn = (FIRST ? g[k] : g[k] * gate[j][k]) * ww[j][k];
                    if (on[j]) {
                        sums[0] = __builtin_fmaf(u, u, sums[0]);
                        sums[1] = __builtin_fmaf(dn, u, sums[1]);
                    }
                }
                if constexpr (!KEEP) {
                    hold_raw(ro[j]);
                    hold_raw(rz[j]);
                    hold_raw(rg[j]);
                }
            }
            team.sum(sums);
            const float q = inv_rms(team, mean, sums[0], [&](auto f) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if constexpr (FIRST && !KEEP)
                        open(j);
                    float v[U];
                    Unit<O, U>::to_float(ro[j], v);
                    if (on[j])
#pragma unroll
                        for (int k = 0; k < U; ++k)
                            f(FIRST ? v[k] * gate[j][k] : v[k]);
                }
            });
            const float back = q * q * (sums[1] * mean.inv_n);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if constexpr (!KEEP) {
                    weigh(j);
                    open(j);
                }
                float v[U], g[U], a[U], b[U];
                Unit<O, U>::to_float(ro[j], v);
                Unit<Act, U>::to_float(rg[j], g);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const float u = FIRST ? v[k] * gate[j][k] : v[k];
                    const float dn = FIRST ? g[k] : g[k] * gate[j][k];
                    const float n = u * q;
                    sw[j][k] = __builtin_fmaf(dn, n, sw[j][k]);
                    const float du = q * (dn * ww[j][k] - u * back);
                    a[k] = FIRST ? du * gate[j][k] : du;
                    b[k] = (FIRST ? du * v[k] : g[k] * n * ww[j][k]) * slope[j][k];
                }
                if (on[j]) {
                    Unit<O, U>::store(spot(dov + base, c[j]), a);
                    Unit<Act, U>::store(spot(dz + row * dz_pitch + static_cast<int64_t>(h) * D, c[j]), b);
                }
            }
        }
    if (w_step == 0) {
        write_part<LPR, U, NV>(team, sw, D, lds, parts + static_cast<int64_t>(blockIdx.x) * D);
    } else if (first < step) {
        float* part = parts + (first * H + h) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (on[j])
#pragma unroll
                for (int k = 0; k < U; ++k)
                    part[c[j] + k] = sw[j][k];
    }
}

// ------------------------------------------------------------ launches

// Lanes of a team and units per lane for rows of n units of U values: the smallest part
// of a wave that holds a row, or a workgroup.  Units of 4 take a lane each up to 1,024
// (8,192 rows of 5,120, fp32 stream: 94 us at 640 lanes of 2, 109 at 320 of 4); units of
// 8 two to a lane above 512, which leaves more rows to a CU (bf16 stream: 74 us at 320
// lanes of 2, 76-85 at 640 of 1), but not where the rows are too few to fill the chip
// (one unit and two, rows of 5,120: 64 rows 3.9 and 4.6 us, 512 6.2 and 6.6, 768 9.0 and
// 8.0, 1,024 10.8 and 8.6, 8,192 64 and 58; of 4,608: 768 6.7 and 8.0, 1,024 9.1 and 8.5,
// 8,192 52 and 54; gated norm of one head, 1,024 and 8,192 of 4,608: 7.5 and 6.3, 40 and
// 38; more than 8,192 values need two anyway) and not in a gradient, whose sums are per
// lane (gated norm, training step of 8,192 rows of 5,120 in bf16: 167 us with two, 157
// with one).
struct Shape {
    int lpr, nv, threads;
};
constexpr int64_t kManyRows = 1024;
inline Shape shape_of(int n, bool pairs) {
    for (int lpr = 4; lpr <= 64; lpr *= 2)
        if (n <= lpr)
            return {lpr, 1, 256};
    int nv = pairs && n > 512 ? 2 : 1;
    while (n > 1024 * nv)
        nv *= 2;
    const int per = (n + nv - 1) / nv;
    return {0, nv, (per + 63) / 64 * 64};
}

template <int U, typename F>
static hipError_t with_shape(const Shape& s, F f) {
    switch (s.lpr) {
        case 4: return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
        case 8: return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
        case 16: return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
        case 32: return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
        case 64: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
        default: break;
    }
    if (s.nv == 1)
        return f(std::integral_constant<int, 0>(), std::integral_constant<int, 1>());
    if constexpr (U == 8) {   // 1,024 lanes of 2 units of 8 hold the widest row
        return f(std::integral_constant<int, 0>(), std::integral_constant<int, 2>());
    } else {
        if (s.nv == 2)
            return f(std::integral_constant<int, 0>(), std::integral_constant<int, 2>());
        return f(std::integral_constant<int, 0>(), std::integral_constant<int, 4>());
    }
}

constexpr int64_t kBlocks = 1 << 16;         // forward workgroups; longer calls loop

// Values to a unit in a residual norm's gradient, of bf16 too: half the registers of 8 and
// twice the lanes to a row.  bf16 stream with w_post, 4 against 8: 8,192 rows of 2,048 48
// and 56 us, 3,161 of 8,680 153 and 352, 2,000 of 12,000 130 and 270 (units of 8 spill
// there); where one unit of 8 to a lane holds a row, units of 8 are the faster ones: 8,192
// of 4,096 98 and 88, of 5,120 154 and 110.
constexpr int kBackUnit = 4;
constexpr int64_t kGatedBlocks = 768;        // workgroups of a gated norm's gradient, each with its own weight sums

// Workgroups of a residual norm's gradient: what the chip holds, since each leaves its own
// weight sums behind.  At about 80 registers to a lane that is 20 waves to a CU; of rows
// with several units to a lane one workgroup, for the 64 or 128 KB of sums in its LDS
// (8,192 rows of 4,096, 1,024 lanes: 98 us with 256 workgroups, 103 with 512; 3,161 of
// 8,680: 153 and 165).
inline int64_t back_blocks(int64_t rows, const Shape& sh) {
    const int teams = sh.lpr ? sh.threads / sh.lpr : 1;
    const int64_t need = (rows + teams - 1) / teams, most = 256 * (sh.nv == 1 ? 1280 / sh.threads : 1);
    return need < most ? need : most;
}

template <typename Act, typename Res>
static hipError_t residual_cfg(const ResidualNorm& a, hipStream_t s) {
    constexpr int U = unit_of<Act, Res>();
    const Shape sh = shape_of(a.W / U, U == 8 && a.rows >= kManyRows);
    const int teams = sh.lpr ? sh.threads / sh.lpr : 1;
    const int64_t need = (a.rows + teams - 1) / teams;
    const dim3 grid(static_cast<unsigned>(need < kBlocks ? need : kBlocks)), block(sh.threads);
    return with_shape<U>(sh, [&](auto lpr, auto nv) {
        auto go = [&](auto post) {
            hipLaunchKernelGGL((residual_norm_kernel<Act, Res, U, lpr(), nv(), post()>), grid, block, 0, s,
                               static_cast<const Res*>(a.residual), static_cast<const Act*>(a.delta), a.scale, a.post,
                               a.w, static_cast<Res*>(a.out), static_cast<Act*>(a.y), a.rows, a.W, Mean(a.W, a.eps));
            return hipGetLastError();
        };
        return a.post ? go(std::true_type()) : go(std::false_type());
    });
}

template <typename Act, typename Res>
static hipError_t residual_back_cfg(const ResidualNormGrad& a, void* ws, hipStream_t s) {
    constexpr int U = kBackUnit;
    const Shape sh = shape_of(a.W / U, false);
    const int64_t blocks = back_blocks(a.rows, sh);
    float* parts = static_cast<float*>(ws);
    hipError_t e = with_shape<U>(sh, [&](auto lpr, auto nv) {
        auto go = [&](auto post) {
            hipLaunchKernelGGL((residual_norm_backward_kernel<Act, Res, U, lpr(), nv(), post()>),
                               dim3(static_cast<unsigned>(blocks)), dim3(sh.threads), 0, s,
                               static_cast<const Res*>(a.stream), static_cast<const Act*>(a.delta), a.scale, a.post,
                               a.w, static_cast<const Act*>(a.dy), static_cast<const Res*>(a.ds),
                               static_cast<Res*>(a.dres), static_cast<Act*>(a.ddelta), parts, a.rows, a.W,
                               Mean(a.W, a.eps));
            return hipGetLastError();
        };
        return a.post ? go(std::true_type()) : go(std::false_type());
    });
    if (e != hipSuccess)
        return e;
    const Sums sums{{a.dw, a.dscale, a.dpost}};
    hipLaunchKernelGGL(part_sum_kernel, dim3(sum_blocks(a.W), a.dpost ? 3 : a.dscale ? 2 : 1), dim3(1024), 0, s, parts,
                       sums, static_cast<int>(blocks), a.W);
    return hipGetLastError();
}

template <typename O, typename Act>
static hipError_t gated_cfg(const GatedNorm& a, hipStream_t s) {
    constexpr int U = unit_of<O, Act>();
    const Shape sh = shape_of(a.D / U, U == 8 && a.rows * a.H >= kManyRows);
    const int teams = sh.lpr ? sh.threads / sh.lpr : 1;
    const int64_t items = a.rows * a.H, need = (items + teams - 1) / teams;
    const dim3 grid(static_cast<unsigned>(need < kBlocks ? need : kBlocks)), block(sh.threads);
    return with_shape<U>(sh, [&](auto lpr, auto nv) {
        auto go = [&](auto first) {
            hipLaunchKernelGGL((gated_norm_kernel<O, Act, U, lpr(), nv(), first()>), grid, block, 0, s,
                               static_cast<const O*>(a.o), static_cast<const Act*>(a.z), a.w, static_cast<Act*>(a.y),
                               items, a.H, a.D, a.z_pitch, a.per_head ? a.D : 0, Mean(a.D, a.eps));
            return hipGetLastError();
        };
        return a.first ? go(std::true_type()) : go(std::false_type());
    });
}

// Workgroups of a gated norm's gradient and the rows that are walked side by side.
struct GatedPlan {
    int64_t blocks, step;
};
inline GatedPlan gated_plan(int64_t rows, int H, int teams) {
    int64_t step = kGatedBlocks * teams / H;
    step = step < 1 ? 1 : step > rows ? rows : step;
    return {(step * H + teams - 1) / teams, step};
}

template <typename O, typename Act>
static hipError_t gated_back_cfg(const GatedNorm& a, const GatedNormGrad& g, void* ws, hipStream_t s) {
    constexpr int U = unit_of<O, Act>();
    const Shape sh = shape_of(a.D / U, false);
    const int teams = sh.lpr ? sh.threads / sh.lpr : 1;
    const GatedPlan plan = gated_plan(a.rows, a.H, teams);
    float* parts = static_cast<float*>(ws);
    hipError_t e = with_shape<U>(sh, [&](auto lpr, auto nv) {
        auto go = [&](auto first) {
            hipLaunchKernelGGL((gated_norm_backward_kernel<O, Act, U, lpr(), nv(), first()>),
                               dim3(static_cast<unsigned>(plan.blocks)), dim3(sh.threads), 0, s,
                               static_cast<const O*>(a.o), static_cast<const Act*>(a.z), a.w,
                               static_cast<const Act*>(g.dy), static_cast<O*>(g.dov), static_cast<Act*>(g.dz), parts,
                               a.rows, a.H, a.D, plan.step, a.z_pitch, g.dz_pitch, a.per_head ? a.D : 0,
                               Mean(a.D, a.eps));
            return hipGetLastError();
        };
        return a.first ? go(std::true_type()) : go(std::false_type());
    });
    if (e != hipSuccess)
        return e;
    const int cols = a.per_head ? a.H * a.D : a.D;
    hipLaunchKernelGGL(part_sum_kernel, dim3(sum_blocks(cols), 1), dim3(1024), 0, s, parts, Sums{{g.dw, nullptr, nullptr}},
                       static_cast<int>(a.per_head ? plan.step : plan.blocks), cols);
    return hipGetLastError();
}

}  // namespace norm

size_t residual_norm_back_ws_bytes(int64_t rows, int W) {
    return static_cast<size_t>(norm::kMaxSums) * norm::back_blocks(rows, norm::shape_of(W / norm::kBackUnit, false)) * W *
           sizeof(float);
}

// The larger of the two layouts over the units of either type of o.
size_t gated_norm_back_ws_bytes(int64_t rows, int H, int D) {
    size_t most = 0;
    for (int U = 4; U <= 8; U += 4) {
        const norm::Shape sh = norm::shape_of(D / U, false);
        const norm::GatedPlan plan = norm::gated_plan(rows, H, sh.lpr ? sh.threads / sh.lpr : 1);
        const size_t shared = static_cast<size_t>(plan.blocks) * D, each = static_cast<size_t>(plan.step) * H * D;
        most = most > shared ? most : shared;
        most = most > each ? most : each;
    }
    return most * sizeof(float);
}

hipError_t launch_residual_norm(const ResidualNorm& a, hipStream_t s) {
    if (!a.act_bf16)
        return norm::residual_cfg<float, float>(a, s);
    return a.res_bf16 ? norm::residual_cfg<uint16_t, uint16_t>(a, s) : norm::residual_cfg<uint16_t, float>(a, s);
}

hipError_t launch_residual_norm_backward(const ResidualNormGrad& a, void* ws, hipStream_t s) {
    if (!a.act_bf16)
        return norm::residual_back_cfg<float, float>(a, ws, s);
    return a.res_bf16 ? norm::residual_back_cfg<uint16_t, uint16_t>(a, ws, s)
                      : norm::residual_back_cfg<uint16_t, float>(a, ws, s);
}

hipError_t launch_gated_norm(const GatedNorm& a, hipStream_t s) {
    if (!a.act_bf16)
        return norm::gated_cfg<float, float>(a, s);
    return a.o_bf16 ? norm::gated_cfg<uint16_t, uint16_t>(a, s) : norm::gated_cfg<float, uint16_t>(a, s);
}

hipError_t launch_gated_norm_backward(const GatedNorm& a, const GatedNormGrad& g, void* ws, hipStream_t s) {
    if (!a.act_bf16)
        return norm::gated_back_cfg<float, float>(a, g, ws, s);
    return a.o_bf16 ? norm::gated_back_cfg<uint16_t, uint16_t>(a, g, ws, s)
                    : norm::gated_back_cfg<float, uint16_t>(a, g, ws, s);
}

}  // namespace gdn
