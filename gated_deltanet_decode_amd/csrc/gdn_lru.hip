// gdn_lru.hip -- the gated linear recurrent layer: one token, prompts, and the
// gradient of a prompt.
//
// Per channel, with rate = min(A, 0), la = rate * sigmoid(r), a = exp(la),
// m = sqrt(1 - a^2):   h <- a h + m sigmoid(i) x,   y = h (times SiLU(z)).
//
// A step is an affine map h -> a h + b, and two of them compose to another, so
// a tile of tokens is first reduced to one map per lane, the maps of the lanes
// before are composed, and each lane then walks its own tokens from the state
// that enters it.  The gradient runs the same way from the other end: with
// e_t = dy_t SiLU(z_t), the gradient of h_t is G_t = e_t + K_{t+1} and
// K_t = a_t G_t is passed on to the token before.
#include "gdn.h"
#include "gdn_lru.hpp"

namespace gdn {
namespace lru {

// ------------------------------------------------------------ one token

template <typename Act, bool GATE>
__global__ __launch_bounds__(256) void lru_token_kernel(float* __restrict__ state, const Act* __restrict__ x,
                                                        const Act* __restrict__ r, const Act* __restrict__ i,
                                                        const float* __restrict__ A, const Act* __restrict__ z,
                                                        Act* __restrict__ y, int W, Pitches p) {
    using Q = Quad<Act>;
    const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= W)
        return;
    const int64_t b = blockIdx.y;
    const typename Q::raw rr = Q::load(r + b * p.r + c), ri = Q::load(i + b * p.i + c), rx = Q::load(x + b * p.x + c);
    const float4 rate4 = *reinterpret_cast<const float4*>(A + c);
    float4* hp = reinterpret_cast<float4*>(state + b * W + c);
    const float4 h4 = *hp;
    typename Q::raw rz;
    if constexpr (GATE)
        rz = Q::load(z + b * p.z + c);
    float fx[4], fr[4], fi[4], fz[4], h[4] = {h4.x, h4.y, h4.z, h4.w}, out[4];
    const float A4[4] = {rate4.x, rate4.y, rate4.z, rate4.w};
    Q::to_float(rx, fx);
    Q::to_float(rr, fr);
    Q::to_float(ri, fi);
    if constexpr (GATE)
        Q::to_float(rz, fz);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, v;
        step(fx[k], fr[k], fi[k], rate2(A4[k]), a, v);
        h[k] = __builtin_fmaf(a, h[k], v);
        out[k] = GATE ? h[k] * silu(fz[k]) : h[k];
    }
    *hp = make_float4(h[0], h[1], h[2], h[3]);
    Q::store(y + b * p.y + c, pack(out, Act()));
}

// ------------------------------------------------------------ prompts
//
// A tile is 64 channels (16 lanes of 4) by 32 groups of N consecutive tokens, 4
// groups to a wave, and one workgroup's work.  The tiles of 64 channels of a
// sequence form a chain along the tokens.  Every tile reads its inputs once and
// keeps a and v in registers; it announces its own map as soon as that is known,
// then gathers the maps of the tiles before it, back to one whose leaving state
// is known already, eight of them at a time (one to a wave), and announces its
// own leaving state.  So the chain costs one exchange of 8 bytes per channel and
// tile, and inputs are not read a second time.
//
// A workgroup takes its tile from a counter, in the order of the chains' tokens:
// whoever holds a tile, all tiles before it are held by workgroups that already
// run and that announce their maps without waiting for anyone.  So every wait
// ends.  An announcement is one relaxed atomic word that is its own flag: the
// words are filled with ones, which no map and no state is (NaNs are made
// canonical), before the kernel starts.

template <typename Act, int N, bool GATE, bool CHAIN>
__global__ __launch_bounds__(kThreads, 4) void lru_scan_kernel(
    float* __restrict__ state, const Act* __restrict__ x, const Act* __restrict__ r, const Act* __restrict__ i,
    const float* __restrict__ A, const Act* __restrict__ z, const int32_t* __restrict__ lengths, Act* __restrict__ y,
    float* __restrict__ saved, int32_t* __restrict__ status, int T, int W, int blocks, int chains, int segs, Chain ch,
    Pitches p) {
    using Q = Quad<Act>;
    constexpr int L = N * kGroups;
    __shared__ Exchange ex;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane & 15, group = wave * 4 + (lane >> 4);
    const int tile = CHAIN ? take_tile(ch, ex) : blockIdx.x;
    if (tile >= chains * segs)
        return;
    const int chain = tile % chains, seg = tile / chains;
    const int b = chain / blocks, c_block = (chain % blocks) * kChannels;
    const bool on = c_block + q * 4 < W;
    const int c = on ? c_block + q * 4 : W - 4;
    const int n = lengths ? lengths[b] : T;
    const bool bad = n < 0 || n > T;
    if (status && threadIdx.x == 0 && seg == 0 && c_block == 0)
        status[b] = bad ? GDN_ERR_INDEX : GDN_OK;
    const int live = bad ? 0 : n - seg * L;   // tokens of the tile and behind it
    if (live <= 0)
        return;
    const int64_t row0 = static_cast<int64_t>(b) * T + seg * L;
    const float4 rate4 = *reinterpret_cast<const float4*>(A + c);
    const float rt[4] = {rate2(rate4.x), rate2(rate4.y), rate2(rate4.z), rate2(rate4.w)};

    const int t0 = group * N;
    float a[N][4], v[N][4];
    float am[4] = {1, 1, 1, 1}, hm[4] = {0, 0, 0, 0};   // the lane's map
    typename Q::raw rz[N];
    {
        typename Q::raw rx[N], rr[N], ri[N];
        const Rows<Act> xs(x, row0, p.x, c), rs(r, row0, p.r, c), is(i, row0, p.i, c);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int t = min(t0 + j, live - 1);
            rr[j] = rs.load(t);
            ri[j] = is.load(t);
            rx[j] = xs.load(t);
        }
        if constexpr (GATE) {
            const Rows<Act> zs(z, row0, p.z, c);
#pragma unroll
            for (int j = 0; j < N; ++j)
                rz[j] = zs.load(min(t0 + j, live - 1));
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float fx[4], fr[4], fi[4];
            Q::to_float(rx[j], fx);
            Q::to_float(rr[j], fr);
            Q::to_float(ri[j], fi);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                step(fx[k], fr[k], fi[k], rt[k], a[j][k], v[j][k]);
                if (t0 + j >= live) {
                    a[j][k] = 1.0f;
                    v[j][k] = 0.0f;
                }
                hm[k] = __builtin_fmaf(a[j][k], hm[k], v[j][k]);
                am[k] *= a[j][k];
            }
        }
    }
    scan_forward(lane, am, hm);
    if (lane >= 48) {
        ex.maps[wave][0][q] = make_float4(am[0], am[1], am[2], am[3]);
        ex.maps[wave][1][q] = make_float4(hm[0], hm[1], hm[2], hm[3]);
    }
    shift_forward(lane, am, hm);
    __syncthreads();

    // the state that enters the tile, and the one that leaves it (one channel to a lane of the first wave)
    const bool last = live <= L;
    float h[4];
    {
        float at = 1.0f, ht = 0.0f;
        const int mine = c_block + lane < W ? c_block + lane : W - 1;
        if (wave == 0) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float wa = ex.map(w, 0)[lane], wh = ex.map(w, 1)[lane];
                ht = __builtin_fmaf(wa, ht, wh);
                at *= wa;
            }
            if (CHAIN && !last && seg > 0)
                ch.announce_map(tile, lane, at, ht);
        }
        float* first = state + static_cast<int64_t>(b) * W;
        float enter = gather<CHAIN>(ch, ex, tile, chains, seg, first + mine, h);
        if (wave == 0) {
            const float leave = __builtin_fmaf(at, enter, ht);
            if (!last)
                ch.announce_state(tile, lane, leave);
            else if (c_block + lane < W)
                first[mine] = leave;
        }
    }
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w)
        if (w < wave)
            compose(h, ex.maps[w][0][q], ex.maps[w][1][q]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = __builtin_fmaf(am[k], h[k], hm[k]);
    if (saved && on && (seg * L + t0) % kSaveStep == 0 && t0 < live) {
        const int marks = (T + kSaveStep - 1) / kSaveStep;
        *reinterpret_cast<float4*>(saved + (static_cast<int64_t>(b) * marks + (seg * L + t0) / kSaveStep) * W + c) =
            make_float4(h[0], h[1], h[2], h[3]);
    }
    const Rows<Act> ys(y, row0, p.y, c);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float out[4], fz[4];
        if constexpr (GATE)
            Q::to_float(rz[j], fz);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = __builtin_fmaf(a[j][k], h[k], v[j][k]);
            out[k] = GATE ? h[k] * silu(fz[k]) : h[k];
        }
        if (on && t0 + j < live)
            ys.store(t0 + j, pack(out, Act()));
    }
}

// Ones in every announcement and 0 in the counter, ahead of a chained kernel.
__global__ __launch_bounds__(256) void lru_clear_kernel(uint4* __restrict__ words, int64_t n, unsigned* __restrict__ next) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; k < n; k += step)
        words[k] = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *next = 0;
}

// ------------------------------------------------------------ the gradient

template <typename Act, int N, bool GATE>
__global__ __launch_bounds__(kThreads) void lru_backward_kernel(
    const Act* __restrict__ x, const Act* __restrict__ r, const Act* __restrict__ i, const float* __restrict__ A,
    const Act* __restrict__ z, const int32_t* __restrict__ lengths, const float* __restrict__ saved,
    const Act* __restrict__ dy, const float* __restrict__ dstate, Act* __restrict__ dx, Act* __restrict__ dr,
    Act* __restrict__ di, Act* __restrict__ dz, float* __restrict__ dstate0, float* __restrict__ parts,
    int32_t* __restrict__ status, int T, int W, int blocks, Pitches p, Pitches gp) {
    using Q = Quad<Act>;
    constexpr int L = N * kGroups;
    static_assert(L == kSaveStep, "a tile starts where a state was saved");
    __shared__ float4 maps[2][kWaves][3][16];
    __shared__ float4 sums[2][kWaves][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane & 15, group = wave * 4 + (lane >> 4);
    const int b = blockIdx.x / blocks, c0 = (blockIdx.x % blocks) * kChannels + q * 4;
    const bool on = c0 < W;
    const int c = on ? c0 : W - 4;
    const int len = lengths ? lengths[b] : T;
    const bool bad = len < 0 || len > T;
    const int n = bad ? 0 : len;
    if (status && threadIdx.x == 0 && blockIdx.x % blocks == 0)
        status[b] = bad ? GDN_ERR_INDEX : GDN_OK;
    const int64_t row0 = static_cast<int64_t>(b) * T;
    x += row0 * p.x + c;
    r += row0 * p.r + c;
    i += row0 * p.i + c;
    dy += row0 * p.y + c;
    dx += row0 * gp.x + c;
    dr += row0 * gp.r + c;
    di += row0 * gp.i + c;
    if constexpr (GATE) {
        z += row0 * p.z + c;
        dz += row0 * gp.z + c;
    }
    const float4 A4 = *reinterpret_cast<const float4*>(A + c);
    const float rate[4] = {rate_of(A4.x), rate_of(A4.y), rate_of(A4.z), rate_of(A4.w)};
    float carry[4] = {0, 0, 0, 0};
    if (dstate) {
        const float4 g = *reinterpret_cast<const float4*>(dstate + static_cast<int64_t>(b) * W + c);
        carry[0] = g.x, carry[1] = g.y, carry[2] = g.z, carry[3] = g.w;
    }
    const int marks = (T + kSaveStep - 1) / kSaveStep;
    for (int seg = marks - 1; seg >= 0; --seg) {
        const int t0 = seg * L + group * N;
        float* part = parts + (static_cast<int64_t>(b) * marks + seg) * W + c;
        if (seg * L >= n) {   // behind the sequence's end: gradients of what was not read
            if (on) {
                const float zero[4] = {0, 0, 0, 0};
                for (int j = 0; j < N; ++j) {
                    const int64_t t = t0 + j;
                    if (t < T && !bad) {
                        Q::store(dx + t * gp.x, pack(zero, Act()));
                        Q::store(dr + t * gp.r, pack(zero, Act()));
                        Q::store(di + t * gp.i, pack(zero, Act()));
                        if constexpr (GATE)
                            Q::store(dz + t * gp.z, pack(zero, Act()));
                    }
                }
                if (group == 0)
                    *reinterpret_cast<float4*>(part) = make_float4(0, 0, 0, 0);
            }
            continue;
        }
        float fx[N][4], a[N][4], m[N][4], im[N][4], rho[N][4], drho[N][4], gi[N][4], dgi[N][4], v[N][4], e[N][4], fdy[N][4],
            sz[N][4], dsz[N][4];
        float am[4] = {1, 1, 1, 1}, hm[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t t = min(t0 + j, n - 1);
            float fr[4], fi[4], fz[4];
            Q::to_float(Q::load(x + t * p.x), fx[j]);
            Q::to_float(Q::load(r + t * p.r), fr);
            Q::to_float(Q::load(i + t * p.i), fi);
            Q::to_float(Q::load(dy + t * p.y), fdy[j]);
            if constexpr (GATE)
                Q::to_float(Q::load(z + t * p.z), fz);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sigmoid_slope(fr[k], rho[j][k], drho[j][k]);
                sigmoid_slope(fi[k], gi[j][k], dgi[j][k]);
                decay(rate[k] * kLog2e * rho[j][k], a[j][k], m[j][k], im[j][k]);
                v[j][k] = m[j][k] * gi[j][k] * fx[j][k];
                if constexpr (GATE) {
                    silu_slope(fz[k], sz[j][k], dsz[j][k]);
                    e[j][k] = fdy[j][k] * sz[j][k];
                } else {
                    e[j][k] = fdy[j][k];
                }
                if (t0 + j >= n) {
                    a[j][k] = 1.0f;
                    v[j][k] = e[j][k] = 0.0f;
                }
                hm[k] = __builtin_fmaf(a[j][k], hm[k], v[j][k]);
                am[k] *= a[j][k];
            }
        }
        float ar[4] = {am[0], am[1], am[2], am[3]}, km[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = N - 1; j >= 0; --j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                km[k] = a[j][k] * (e[j][k] + km[k]);
        scan_forward(lane, am, hm);
        scan_reverse(lane, ar, km);
        if (lane >= 48) {
            maps[seg & 1][wave][0][q] = make_float4(am[0], am[1], am[2], am[3]);
            maps[seg & 1][wave][1][q] = make_float4(hm[0], hm[1], hm[2], hm[3]);
        }
        if (lane < 16)
            maps[seg & 1][wave][2][q] = make_float4(km[0], km[1], km[2], km[3]);
        shift_forward(lane, am, hm);
        shift_reverse(lane, ar, km);
        __syncthreads();
        const float4 h4 = *reinterpret_cast<const float4*>(saved + (static_cast<int64_t>(b) * marks + seg) * W + c);
        float h[4] = {h4.x, h4.y, h4.z, h4.w}, K[4] = {carry[0], carry[1], carry[2], carry[3]};
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (w < wave)
                compose(h, maps[seg & 1][w][0][q], maps[seg & 1][w][1][q]);
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
            const float4 ma = maps[seg & 1][w][0][q], mk = maps[seg & 1][w][2][q];
            compose(carry, ma, mk);
            if (w > wave)
                compose(K, ma, mk);
        }
        float before[N][4], after[N][4], dA[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = __builtin_fmaf(am[k], h[k], hm[k]);
            K[k] = __builtin_fmaf(ar[k], K[k], km[k]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                before[j][k] = h[k];
                h[k] = __builtin_fmaf(a[j][k], h[k], v[j][k]);
                after[j][k] = h[k];
            }
#pragma unroll
        for (int j = N - 1; j >= 0; --j) {
            float ox[4], orr[4], oi[4], oz[4];
            const bool live = t0 + j < n;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float G = e[j][k] + K[k];
                K[k] = a[j][k] * G;
                const float gx = gi[j][k] * fx[j][k];
                const float dla = G * (a[j][k] * before[j][k] - a[j][k] * a[j][k] * im[j][k] * gx);
                ox[k] = live ? G * m[j][k] * gi[j][k] : 0.0f;
                oi[k] = live ? G * m[j][k] * fx[j][k] * dgi[j][k] : 0.0f;
                orr[k] = live ? dla * rate[k] * drho[j][k] : 0.0f;
                if constexpr (GATE)
                    oz[k] = live ? fdy[j][k] * after[j][k] * dsz[j][k] : 0.0f;
                dA[k] += live ? dla * rho[j][k] : 0.0f;
            }
            const int64_t t = t0 + j;
            if (on && t < T) {
                Q::store(dx + t * gp.x, pack(ox, Act()));
                Q::store(dr + t * gp.r, pack(orr, Act()));
                Q::store(di + t * gp.i, pack(oi, Act()));
                if constexpr (GATE)
                    Q::store(dz + t * gp.z, pack(oz, Act()));
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            dA[k] += __shfl_xor(dA[k], 16);
            dA[k] += __shfl_xor(dA[k], 32);
        }
        if (lane < 16)
            sums[seg & 1][wave][q] = make_float4(dA[0], dA[1], dA[2], dA[3]);
        __syncthreads();
        if (on && group == 0) {
            float s[4] = {0, 0, 0, 0};
            for (int w = 0; w < kWaves; ++w) {
                const float4 u = sums[seg & 1][w][q];
                s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w;
            }
            *reinterpret_cast<float4*>(part) = make_float4(s[0], s[1], s[2], s[3]);
        }
    }
    if (on && group == 0 && !bad && dstate0)
        *reinterpret_cast<float4*>(dstate0 + static_cast<int64_t>(b) * W + c) =
            make_float4(carry[0], carry[1], carry[2], carry[3]);
}

// dA from the tiles' sums, in a fixed order: 4 waves take every fourth row each.
__global__ __launch_bounds__(256) void lru_rate_kernel(const float* __restrict__ parts, const float* __restrict__ A,
                                                       float* __restrict__ dA, int rows, int W) {
    __shared__ float sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < W)
        for (int row = wave; row < rows; row += 4)
            s += parts[static_cast<int64_t>(row) * W + c];
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < W)
        dA[c] = A[c] < 0.0f ? (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]) : 0.0f;
}

template <typename Act, bool GATE>
static hipError_t token_cfg(const LruGeo& g, const LruArgs& a, hipStream_t s) {
    const dim3 grid((g.W / 4 + 255) / 256, g.B);
    hipLaunchKernelGGL((lru_token_kernel<Act, GATE>), grid, dim3(256), 0, s, a.state, static_cast<const Act*>(a.x),
                       static_cast<const Act*>(a.r), static_cast<const Act*>(a.i), a.A, static_cast<const Act*>(a.z),
                       static_cast<Act*>(a.y), g.W, g.p);
    return hipGetLastError();
}

// The workspace of a chained call: 256 bytes with the counter, then a word of 8
// bytes (map) and one of 4 (state) per channel and tile.
// Tokens of a lane's group in a chained prompt: what its registers hold.
constexpr int tokens_of(bool bf16) { return bf16 ? 8 : 4; }
inline int64_t scan_tiles(const LruGeo& g, int T) {
    const int L = tokens_of(g.bf16) * kGroups;
    return static_cast<int64_t>(g.B) * ((g.W + kChannels - 1) / kChannels) * ((T + L - 1) / L);
}
inline size_t chain_bytes(int64_t tiles) { return 256 + static_cast<size_t>(tiles) * kChannels * 12; }

static hipError_t clear_chain(void* ws, int64_t tiles, Chain& ch, hipStream_t s) {
    char* p = static_cast<char*>(ws);
    ch.next = reinterpret_cast<unsigned*>(p);
    ch.maps = reinterpret_cast<uint64_t*>(p + 256);
    ch.states = reinterpret_cast<uint32_t*>(p + 256 + tiles * kChannels * 8);
    const int64_t words = tiles * kChannels * 12 / 16;
    const int64_t grid = (words + 1023) / 1024;
    hipLaunchKernelGGL(lru_clear_kernel, dim3(static_cast<unsigned>(grid < 2048 ? grid : 2048)), dim3(256), 0, s,
                       reinterpret_cast<uint4*>(p + 256), words, ch.next);
    return hipGetLastError();
}

template <typename Act, int N, bool GATE, bool CHAIN>
static hipError_t scan_launch(const LruGeo& g, const LruArgs& a, int T, const int32_t* lengths, float* saved,
                              int32_t* status, const Chain& ch, hipStream_t s) {
    const int blocks = (g.W + kChannels - 1) / kChannels, segs = CHAIN ? (T + N * kGroups - 1) / (N * kGroups) : 1;
    hipLaunchKernelGGL((lru_scan_kernel<Act, N, GATE, CHAIN>), dim3(static_cast<unsigned>(g.B) * blocks * segs),
                       dim3(kThreads), 0, s, a.state, static_cast<const Act*>(a.x), static_cast<const Act*>(a.r),
                       static_cast<const Act*>(a.i), a.A, static_cast<const Act*>(a.z), lengths,
                       static_cast<Act*>(a.y), saved, status, T, g.W, blocks, g.B * blocks, segs, ch, g.p);
    return hipGetLastError();
}


template <typename Act, bool GATE>
static hipError_t scan_cfg(const LruGeo& g, const LruArgs& a, int T, const int32_t* lengths, float* saved,
                           int32_t* status, void* ws, hipStream_t s) {
    constexpr int N = tokens_of(sizeof(Act) == 2);
    Chain ch = {};
    if (T <= 2 * kGroups)
        return scan_launch<Act, 2, GATE, false>(g, a, T, lengths, saved, status, ch, s);
    if (T <= 4 * kGroups)
        return scan_launch<Act, 4, GATE, false>(g, a, T, lengths, saved, status, ch, s);
    if (T <= N * kGroups)
        return scan_launch<Act, N, GATE, false>(g, a, T, lengths, saved, status, ch, s);
    const hipError_t e = clear_chain(ws, scan_tiles(g, T), ch, s);
    return e != hipSuccess ? e : scan_launch<Act, N, GATE, true>(g, a, T, lengths, saved, status, ch, s);
}

template <typename Act, bool GATE>
static hipError_t backward_cfg(const LruGeo& g, const LruGrads& a, int T, const int32_t* lengths, int32_t* status,
                               void* ws, hipStream_t s) {
    const int blocks = (g.W + kChannels - 1) / kChannels;
    float* parts = static_cast<float*>(ws);
    hipLaunchKernelGGL((lru_backward_kernel<Act, 4, GATE>), dim3(g.B * blocks), dim3(kThreads), 0, s,
                       static_cast<const Act*>(a.x), static_cast<const Act*>(a.r), static_cast<const Act*>(a.i), a.A,
                       static_cast<const Act*>(a.z), lengths, a.saved, static_cast<const Act*>(a.dy), a.dstate,
                       static_cast<Act*>(a.dx), static_cast<Act*>(a.dr), static_cast<Act*>(a.di),
                       static_cast<Act*>(a.dz), a.dstate0, parts, status, T, g.W, blocks, g.p, g.gp);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int rows = g.B * ((T + kSaveStep - 1) / kSaveStep);
    hipLaunchKernelGGL(lru_rate_kernel, dim3((g.W + 63) / 64), dim3(256), 0, s, parts, a.A, a.dA, rows, g.W);
    return hipGetLastError();
}

}  // namespace lru

hipError_t launch_lru_token(const LruGeo& g, const LruArgs& a, hipStream_t s) {
    if (g.bf16)
        return a.z ? lru::token_cfg<uint16_t, true>(g, a, s) : lru::token_cfg<uint16_t, false>(g, a, s);
    return a.z ? lru::token_cfg<float, true>(g, a, s) : lru::token_cfg<float, false>(g, a, s);
}

size_t lru_saved_bytes(const LruGeo& g, int T) {
    return static_cast<size_t>(g.B) * ((T + lru::kSaveStep - 1) / lru::kSaveStep) * g.W * sizeof(float);
}

size_t lru_prefill_ws_bytes(const LruGeo& g, int T) {
    return T <= lru::tokens_of(g.bf16) * lru::kGroups ? 0 : lru::chain_bytes(lru::scan_tiles(g, T));
}

hipError_t launch_lru_prefill(const LruGeo& g, const LruArgs& a, int T, const int32_t* lengths, float* saved,
                              int32_t* status, void* ws, hipStream_t s) {
    if (g.bf16)
        return a.z ? lru::scan_cfg<uint16_t, true>(g, a, T, lengths, saved, status, ws, s)
                   : lru::scan_cfg<uint16_t, false>(g, a, T, lengths, saved, status, ws, s);
    return a.z ? lru::scan_cfg<float, true>(g, a, T, lengths, saved, status, ws, s)
               : lru::scan_cfg<float, false>(g, a, T, lengths, saved, status, ws, s);
}

size_t lru_backward_ws_bytes(const LruGeo& g, int T) { return lru_saved_bytes(g, T); }

hipError_t launch_lru_backward(const LruGeo& g, const LruGrads& a, int T, const int32_t* lengths, int32_t* status,
                               void* ws, hipStream_t s) {
    if (g.bf16)
        return a.z ? lru::backward_cfg<uint16_t, true>(g, a, T, lengths, status, ws, s)
                   : lru::backward_cfg<uint16_t, false>(g, a, T, lengths, status, ws, s);
    return a.z ? lru::backward_cfg<float, true>(g, a, T, lengths, status, ws, s)
               : lru::backward_cfg<float, false>(g, a, T, lengths, status, ws, s);
}

}  // namespace gdn
