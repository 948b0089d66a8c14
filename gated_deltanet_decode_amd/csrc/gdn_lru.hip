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
//
// Four channels to a lane, everything read once and written once.  Below some 10 MB
// the launch sets the time (one sequence of 5,120 channels 2.3 us, 200 of 4,096, 14.7
// MB, 4.5 us in a trace).

template <typename Act, bool GATE>
__global__ __launch_bounds__(256) void lru_token_kernel(float* __restrict__ state, const Act* __restrict__ x,
                                                        const Act* __restrict__ r, const Act* __restrict__ i,
                                                        const float* __restrict__ A, const Act* __restrict__ z,
                                                        Act* __restrict__ y, unsigned lanes, unsigned per_row, int W,
                                                        Pitches p) {
    using Q = Quad<Act>;
    const unsigned at = blockIdx.x * 256 + threadIdx.x;   // four channels of one sequence
    if (at >= lanes)
        return;
    const int64_t b = at / per_row;
    const int c = static_cast<int>(at % per_row) * 4;
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
// A tile is a block of channels by some tokens, and one workgroup's work.  The tiles
// of a sequence's channels form a chain along the tokens.  Every tile reads its
// inputs once and keeps a and v in registers; it announces its own map as soon as
// that is known, looks at as many tiles before it as it has waves until one of them
// shows the state that leaves it, applies the maps from there, and announces its own
// leaving state.  So the chain costs one word of 8 bytes per channel and tile, and
// inputs are not read a second time.
//
// A workgroup takes its tile from a counter, in the order of the chains' tokens:
// whoever holds a tile, all tiles before it are held by workgroups that already run.
// Maps are announced without waiting, and the first tile of a chain waits for nobody,
// so one after the other shows its state and every wait ends.  An announcement is one
// relaxed atomic word that is its own flag, so that it orders no other memory; the
// words are filled with ones, which no announcement is, before the kernel starts.
// (Workgroups that stay and take one tile after the other hold a tile back while they
// finish another, and its chain with it: 388 against 260 us at 32,768 tokens of 4,096
// channels.)
//
// What bounds it is how HBM takes a tile's rows: a kernel that only moves the same
// pieces of rows takes 268 us where they are 128 bytes, 229 at 256 bytes and 225 at
// 512, against 218 in linear order; without its exponentials this one takes no less,
// without the chain 238 us.  Half a wave to a row (256 bytes in bf16) and 8 tokens to
// a lane keep the registers at 121, two workgroups to a CU.
// Measured: 32,768 tokens of 4,096 channels, z, bf16: 260 us, 5.2 TB/s (a copy of
// 1 GiB runs at 5.2); 4 x 4,096 tokens in fp32: 247 us, 5.4 TB/s.

template <typename Act, int LPC, int WAVES, int N, bool GATE, bool CHAIN>
__global__ __launch_bounds__(WAVES * kWave, 4) void lru_scan_kernel(
    float* __restrict__ state, const Act* __restrict__ x, const Act* __restrict__ r, const Act* __restrict__ i,
    const float* __restrict__ A, const Act* __restrict__ z, const int32_t* __restrict__ lengths, Act* __restrict__ y,
    float* __restrict__ saved, int32_t* __restrict__ status, int T, int W, int blocks, int chains, int segs, Chain ch,
    Pitches p) {
    using Q = Quad<Act>;
    using TL = Tile<LPC, WAVES, N>;
    constexpr int L = TL::kTokens, E = TL::kWords;
    __shared__ Exchange<TL, WAVES, 2> ex;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane % LPC, group = wave * TL::kPerWave + lane / LPC;
    const int tile = CHAIN ? take_tile(ch, ex) : blockIdx.x;
    if (tile >= chains * segs)
        return;
    const int chain = tile % chains, seg = tile / chains;
    const int b = chain / blocks, c_block = (chain % blocks) * TL::kChannels;
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
    const int t0 = group * N;
    const Rows<Act> xs(x, row0, p.x, c), rs(r, row0, p.r, c), is(i, row0, p.i, c), zs(GATE ? z : x, row0, p.z, c);
    typename Q::raw rx[N], rr[N], ri[N], rz[N];
    // z is asked for with the rest in bf16; fp32 has no registers for it until x, r and i are used
    constexpr bool LATE = GATE && sizeof(Act) == 4;
    if (live >= L) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            rr[j] = rs.load(t0, j);
            ri[j] = is.load(t0, j);
            rx[j] = xs.load(t0, j);
        }
        if constexpr (GATE && !LATE)
#pragma unroll
            for (int j = 0; j < N; ++j)
                rz[j] = zs.load(t0, j);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int t = min(t0 + j, live - 1);
            rr[j] = rs.load(t);
            ri[j] = is.load(t);
            rx[j] = xs.load(t);
            if constexpr (GATE && !LATE)
                rz[j] = zs.load(t);
        }
    }
    float* enter = state + static_cast<int64_t>(b) * W;
    const float first = seg == 0 && wave < E ? enter[min(c_block + wave * kWave + lane, W - 1)] : 0.0f;
    const float4 rate4 = *reinterpret_cast<const float4*>(A + c);
    const float rt[4] = {rate2(rate4.x), rate2(rate4.y), rate2(rate4.z), rate2(rate4.w)};

    float a[N][4], v[N][4];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float fx[4], fr[4], fi[4];
        Q::to_float(rx[j], fx);
        Q::to_float(rr[j], fr);
        Q::to_float(ri[j], fi);
#pragma unroll
        for (int k = 0; k < 4; ++k)
        {
            step(fx[k], fr[k], fi[k], rt[k], a[j][k], v[j][k]);
            settle(v[j][k]);
        }
    }
    if (live < L)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t0 + j >= live) {
                    a[j][k] = 1.0f;
                    v[j][k] = 0.0f;
                }
    if constexpr (LATE)
#pragma unroll
        for (int j = 0; j < N; ++j)
            rz[j] = zs.load(min(t0 + j, live - 1));
    float am[4] = {1, 1, 1, 1}, hm[4] = {0, 0, 0, 0}, wa[4], wv[4];   // the lane's map, then the wave's
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hm[k] = __builtin_fmaf(a[j][k], hm[k], v[j][k]);
            am[k] *= a[j][k];
        }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        scan_forward<LPC>(lane, am[k], hm[k], wa[k], wv[k]);
    if (lane >= kWave - LPC) {
        put4(ex.maps[wave][0], q, wa);
        put4(ex.maps[wave][1], q, wv);
    }
    __syncthreads();

    const bool last = live <= L, holds = wave < E;
    const int hc = wave * kWave + lane;   // the channel that the first E waves' lanes hold, of the tile's
    const int64_t word = static_cast<int64_t>(tile) * TL::kChannels + hc;
    float at = 1.0f, ht = 0.0f;           // the tile's map
    if (holds) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            ht = __builtin_fmaf(ex.maps[w][0][hc], ht, ex.maps[w][1][hc]);
            at *= ex.maps[w][0][hc];
        }
        if (CHAIN && !last && seg > 0)
            ch.announce_map(word, at, ht);
    }
    float in = gather<TL, WAVES, CHAIN>(ch, ex, wave, tile, chains, seg, first);
    if (holds) {
        const float leave = __builtin_fmaf(at, in, ht);
        if (!last)
            ch.announce_state(word, leave);
        else if (c_block + hc < W)
            enter[c_block + hc] = leave;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            ex.into[0][w][hc] = in;
            in = __builtin_fmaf(ex.maps[w][0][hc], in, ex.maps[w][1][hc]);
        }
    }
    __syncthreads();
    float h[4];
    get4(ex.into[0][wave], q, h);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = __builtin_fmaf(am[k], h[k], hm[k]);
    const Rows<Act> ys(y, row0, p.y, c);
    const bool whole = live >= L && c_block + TL::kChannels <= W;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (saved && (seg * L + t0 + j) % kSaveStep == 0 && on && t0 + j < live) {
            const int marks = (T + kSaveStep - 1) / kSaveStep;
            *reinterpret_cast<float4*>(saved + (static_cast<int64_t>(b) * marks + (seg * L + t0 + j) / kSaveStep) * W + c) =
                make_float4(h[0], h[1], h[2], h[3]);
        }
        float out[4], fz[4];
        if constexpr (GATE)
            Q::to_float(rz[j], fz);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = __builtin_fmaf(a[j][k], h[k], v[j][k]);
            out[k] = GATE ? h[k] * silu(fz[k]) : h[k];
        }
        if (whole || (on && t0 + j < live))
            ys.store(t0, j, pack(out, Act()));
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
//
// The chains run from the last token to the first.  A tile starts from a state that
// the forward pass saved, so its own h need no chain; what it passes on is K, the
// gradient of the state before its first token, whose map has the same a.  With
// P = a sigmoid(i) x / m, the gradient of la is G (a h' - a^2 sigmoid(i) x / m) =
// K (h' - P) for h' the state before the token, so the two parts of a token's
// decay share one product.  What the outputs need of a token (nine values) stays in
// registers while the chain is waited for, so that its exponentials are taken once;
// that is 72 registers at 2 tokens to a lane.  Each tile's part of dA goes to `parts`.
//
// Nine streams (five in, four out).  Measured, 4 x 4,096 tokens of 4,096 channels
// with z: bf16 280-295 us, 4.2 TB/s; fp32 403 us, 6.0 TB/s.  The arithmetic does not set
// it (270 us without the exponentials in bf16, 399 in fp32), nor the chain (270): a
// bf16 tile has half the bytes under way of an fp32 one, for the same latencies.
// Four tokens to a lane, which doubles them, halve the waves: 297 against 283 us at
// 16 x 1,024 tokens.

template <typename Act, int LPC, int WAVES, int N, bool GATE, bool CHAIN>
__global__ __launch_bounds__(WAVES * kWave, 4) void lru_backward_kernel(
    const Act* __restrict__ x, const Act* __restrict__ r, const Act* __restrict__ i, const float* __restrict__ A,
    const Act* __restrict__ z, const int32_t* __restrict__ lengths, const float* __restrict__ saved,
    const Act* __restrict__ dy, const float* dstate, Act* __restrict__ dx, Act* __restrict__ dr, Act* __restrict__ di,
    Act* __restrict__ dz, float* dstate0, float* __restrict__ parts, int32_t* __restrict__ status, int T, int W,
    int blocks, int chains, int segs, Chain ch, Pitches p, Pitches gp) {
    using Q = Quad<Act>;
    using TL = Tile<LPC, WAVES, N>;
    constexpr int L = TL::kTokens, E = TL::kWords;
    static_assert(L % kSaveStep == 0, "a tile starts where a state was saved");
    __shared__ Exchange<TL, WAVES, 3> ex;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane % LPC, group = wave * TL::kPerWave + lane / LPC;
    const int tile = CHAIN ? take_tile(ch, ex) : blockIdx.x;
    if (tile >= chains * segs)
        return;
    const int chain = tile % chains, seg = segs - 1 - tile / chains;
    const int b = chain / blocks, c_block = (chain % blocks) * TL::kChannels;
    const bool on = c_block + q * 4 < W;
    const int c = on ? c_block + q * 4 : W - 4;
    const int n = lengths ? lengths[b] : T;
    const bool bad = n < 0 || n > T;
    if (status && threadIdx.x == 0 && seg == 0 && c_block == 0)
        status[b] = bad ? GDN_ERR_INDEX : GDN_OK;
    const int64_t row0 = static_cast<int64_t>(b) * T + seg * L;
    const int t0 = group * N, rows = min(T - seg * L, L), live = bad ? 0 : n - seg * L;
    const Rows<Act> xg(dx, row0, gp.x, c), rg(dr, row0, gp.r, c), ig(di, row0, gp.i, c), zg(GATE ? dz : dx, row0, gp.z, c);
    float* part = parts + (static_cast<int64_t>(b) * segs + seg) * W;
    const bool holds = wave < E;
    const int hc = wave * kWave + lane, mine = min(c_block + hc, W - 1);   // the channel that the first E waves' lanes hold
    if (live <= 0) {   // behind the sequence's end: the gradient of what was not read
        const float zero[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (on && !bad && t0 + j < rows) {
                xg.store(t0, j, pack(zero, Act()));
                rg.store(t0, j, pack(zero, Act()));
                ig.store(t0, j, pack(zero, Act()));
                if constexpr (GATE)
                    zg.store(t0, j, pack(zero, Act()));
            }
        if (on && group == 0)
            *reinterpret_cast<float4*>(part + c) = make_float4(0, 0, 0, 0);
        if (seg == 0 && holds && !bad && dstate0 && c_block + hc < W)   // no token at all: the state passes through
            dstate0[static_cast<int64_t>(b) * W + mine] = dstate ? dstate[static_cast<int64_t>(b) * W + mine] : 0.0f;
        return;
    }
    const Rows<Act> xs(x, row0, p.x, c), rs(r, row0, p.r, c), is(i, row0, p.i, c), ds(dy, row0, p.y, c),
        zs(GATE ? z : x, row0, p.z, c);
    typename Q::raw rx[N], rr[N], ri[N], rd[N], rz[N];
    if (live >= L) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            rr[j] = rs.load(t0, j);
            ri[j] = is.load(t0, j);
            rx[j] = xs.load(t0, j);
            rd[j] = ds.load(t0, j);
            if constexpr (GATE)
                rz[j] = zs.load(t0, j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int t = min(t0 + j, live - 1);
            rr[j] = rs.load(t);
            ri[j] = is.load(t);
            rx[j] = xs.load(t);
            rd[j] = ds.load(t);
            if constexpr (GATE)
                rz[j] = zs.load(t);
        }
    }
    const int marks = (T + kSaveStep - 1) / kSaveStep;
    float h0 = holds ? saved[(static_cast<int64_t>(b) * marks + seg * (L / kSaveStep)) * W + mine] : 0.0f;
    const int dist = (n + L - 1) / L - 1 - seg;   // place in the chain: the sequence's last tile is its first
    const float first = dist == 0 && holds && dstate ? dstate[static_cast<int64_t>(b) * W + mine] : 0.0f;
    const float4 A4 = *reinterpret_cast<const float4*>(A + c);
    const float rate[4] = {rate_of(A4.x), rate_of(A4.y), rate_of(A4.z), rate_of(A4.w)};

    // of a token: its map, the output's gradient, and the factors of the outputs
    float a[N][4], v[N][4], eg[N][4], fx[N][4], fi[N][4], fp[N][4], fr[N][4], rho[N][4], fd[N][4];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float x4[4], r4[4], i4[4], d4[4], z4[4];
        Q::to_float(rx[j], x4);
        Q::to_float(rr[j], r4);
        Q::to_float(ri[j], i4);
        Q::to_float(rd[j], d4);
        if constexpr (GATE)
            Q::to_float(rz[j], z4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float slope, g, shut, m, inv;
            sigmoid_slope(r4[k], rho[j][k], slope);
            fr[j][k] = rate[k] * slope;
            decay(rate[k] * kLog2e * rho[j][k], a[j][k], m, inv);
            sigmoid_both(i4[k], g, shut);
            const float gx = g * x4[k];
            v[j][k] = m * gx;
            fx[j][k] = m * g;
            fi[j][k] = v[j][k] * shut;
            fp[j][k] = a[j][k] * inv * gx;
            if constexpr (GATE) {
                float s, ds;
                silu_slope(z4[k], s, ds);
                eg[j][k] = d4[k] * s;
                fd[j][k] = d4[k] * ds;
                settle(fd[j][k]);
            } else {
                eg[j][k] = d4[k];
            }
            settle(v[j][k]);
            settle(eg[j][k]);
            settle(fx[j][k]);
            settle(fi[j][k]);
            settle(fp[j][k]);
            settle(fr[j][k]);
        }
    }
    if (live < L)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t0 + j >= live) {
                    a[j][k] = 1.0f;
                    v[j][k] = eg[j][k] = rho[j][k] = 0.0f;
                }
    float am[4] = {1, 1, 1, 1}, hm[4] = {0, 0, 0, 0}, km[4] = {0, 0, 0, 0}, ar[4], wa[4], wv[4], wk[4];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hm[k] = __builtin_fmaf(a[j][k], hm[k], v[j][k]);
            am[k] *= a[j][k];
        }
#pragma unroll
    for (int j = N - 1; j >= 0; --j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            km[k] = a[j][k] * (eg[j][k] + km[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        ar[k] = am[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        scan_forward<LPC>(lane, am[k], hm[k], wa[k], wv[k]);
        scan_reverse<LPC>(lane, ar[k], km[k], wk[k]);
    }
    if (lane >= kWave - LPC) {
        put4(ex.maps[wave][0], q, wa);
        put4(ex.maps[wave][1], q, wv);
    }
    if (lane < LPC)
        put4(ex.maps[wave][2], q, wk);
    __syncthreads();

    const bool last = seg == 0;
    const int64_t word = static_cast<int64_t>(tile) * TL::kChannels + hc;
    float at = 1.0f, kt = 0.0f;   // the tile's map
    if (holds) {
#pragma unroll
        for (int w = WAVES - 1; w >= 0; --w) {
            kt = __builtin_fmaf(ex.maps[w][0][hc], kt, ex.maps[w][2][hc]);
            at *= ex.maps[w][0][hc];
        }
        if (CHAIN && !last && dist > 0)
            ch.announce_map(word, at, kt);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            ex.into[0][w][hc] = h0;
            h0 = __builtin_fmaf(ex.maps[w][0][hc], h0, ex.maps[w][1][hc]);
        }
    }
    float in = gather<TL, WAVES, CHAIN>(ch, ex, wave, tile, chains, dist, first);
    if (holds) {
        const float leave = __builtin_fmaf(at, in, kt);
        if (!last)
            ch.announce_state(word, leave);
        else if (dstate0 && c_block + hc < W)
            dstate0[static_cast<int64_t>(b) * W + mine] = leave;
#pragma unroll
        for (int w = WAVES - 1; w >= 0; --w) {
            ex.into[1][w][hc] = in;
            in = __builtin_fmaf(ex.maps[w][0][hc], in, ex.maps[w][2][hc]);
        }
    }
    // h before each token, less P
    float h[4], K[4], dA[4] = {0, 0, 0, 0};
    get4(ex.into[0][wave], q, h);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = __builtin_fmaf(am[k], h[k], hm[k]);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            fp[j][k] = h[k] - fp[j][k];
            h[k] = __builtin_fmaf(a[j][k], h[k], v[j][k]);
            if constexpr (GATE)
                fd[j][k] *= h[k];
        }
    __syncthreads();
    get4(ex.into[1][wave], q, K);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        K[k] = __builtin_fmaf(ar[k], K[k], km[k]);
    const bool whole = live >= L && c_block + TL::kChannels <= W;
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
        float ox[4], orr[4], oi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float G = eg[j][k] + K[k];
            K[k] = a[j][k] * G;
            const float dla = K[k] * fp[j][k];
            ox[k] = G * fx[j][k];
            oi[k] = G * fi[j][k];
            orr[k] = dla * fr[j][k];
            dA[k] = __builtin_fmaf(dla, rho[j][k], dA[k]);
        }
        if (whole) {
            xg.store(t0, j, pack(ox, Act()));
            rg.store(t0, j, pack(orr, Act()));
            ig.store(t0, j, pack(oi, Act()));
            if constexpr (GATE)
                zg.store(t0, j, pack(fd[j], Act()));
        } else if (on && t0 + j < rows) {
            const bool dead = t0 + j >= live;
            if (dead)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ox[k] = oi[k] = orr[k] = fd[j][k] = 0.0f;
            xg.store(t0, j, pack(ox, Act()));
            rg.store(t0, j, pack(orr, Act()));
            ig.store(t0, j, pack(oi, Act()));
            if constexpr (GATE)
                zg.store(t0, j, pack(fd[j], Act()));
        }
    }
    // the tile's part of dA: over a wave's groups, then over the waves
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int d = LPC; d < kWave; d *= 2)
            dA[k] += __shfl_xor(dA[k], d);
    if (lane < LPC)
        put4(ex.look[wave][0], q, dA);   // the chain's words have been read
    __syncthreads();
    if (holds && c_block + hc < W) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            s += ex.look[w][0][hc];
        part[c_block + hc] = s;
    }
}

// dA from the tiles' parts, in a fixed order: 16 waves take every 16th row each.
__global__ __launch_bounds__(1024) void lru_rate_kernel(const float* __restrict__ parts, const float* __restrict__ A,
                                                        float* __restrict__ dA, int rows, int W) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < W) {
        const float* p = parts + c;
#pragma unroll 8
        for (int row = wave; row < rows; row += 16)
            s += p[static_cast<int64_t>(row) * W];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < W) {
        float t = 0.0f;
        for (int w = 0; w < 16; ++w)
            t += sums[w][lane];
        dA[c] = A[c] >= 0.0f ? 0.0f : t;
    }
}

template <typename Act, bool GATE>
static hipError_t token_cfg(const LruGeo& g, const LruArgs& a, hipStream_t s) {
    const unsigned per_row = g.W / 4, lanes = g.B * per_row;   // fewer than 2^27: B * ceil(W / 64) < 2^23
    hipLaunchKernelGGL((lru_token_kernel<Act, GATE>), dim3((lanes + 255) / 256), dim3(256), 0, s, a.state,
                       static_cast<const Act*>(a.x), static_cast<const Act*>(a.r), static_cast<const Act*>(a.i), a.A,
                       static_cast<const Act*>(a.z), static_cast<Act*>(a.y), lanes, per_row, g.W, g.p);
    return hipGetLastError();
}

// Tiles of the kernels over prompts.
struct Shape {
    int channels, tokens, blocks, segs;
    int64_t tiles;
};
inline Shape shape_of(const LruGeo& g, int T, int channels, int tokens) {
    Shape s;
    s.channels = channels;
    s.tokens = tokens;
    s.blocks = (g.W + channels - 1) / channels;
    s.segs = (T + tokens - 1) / tokens;
    s.tiles = static_cast<int64_t>(g.B) * s.blocks * s.segs;
    return s;
}

constexpr int kWide = 128;   // channels of a wide tile
constexpr int kScanTokens = 128, kBackTokens = 32;

// Wide tiles (32 lanes to a row) where they are enough for the chip, 64 channels else.
// bf16, wide against narrow: 16 x 256 tokens of 1,024 channels (256 tiles) 16.8 and
// 19.4 us, 1 x 1,024 of 2,560 (160) 15.1 and 15.7.  fp32, whose narrow rows are 256
// bytes already: 1 x 4,096 of 2,560 (640) 56 and 49 us, 8 x 2,500 (3,200) 196 both.
// Up to 256 tokens one narrow tile holds the whole prompt and nothing is chained: 1 x
// 256 of 2,560 9.5 us against 10.9 in two tiles.
inline Shape scan_shape(const LruGeo& g, int T) {
    const Shape s = shape_of(g, T, kWide, kScanTokens);
    if (s.segs > 1 && s.tiles >= (g.bf16 ? 128 : 1024))
        return s;
    return shape_of(g, T, 64, T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : T <= 256 ? 256 : 128);
}
// A wide tile of the gradient has 32 tokens, a narrow one 64, so that narrow chains are
// half as long: 16 x 64 tokens of 4,096 channels (1,024 wide tiles) 31 us wide, 24
// narrow; 1 x 8,192 of 512 (1,024) 68 and 44; 8 x 300 of 2,048 in fp32 (1,280) 42 both;
// 1 x 4,096 of 2,560 (2,560) 67 and 66; 16 x 1,024 of 4,096 (16,384) 278 and 283, 4 x
// 4,096 of 4,096 in fp32 402 and 443.  Between them the count does not tell: 3 x 1,003 of
// 1,544 (1,248) take narrow tiles and 45 us wide, 52 narrow, in fp32 without z 47 and 49.
// At most 64 channels leave half of a wide tile's lanes off: 512 x 512 of 64 165 wide, 95
// narrow; 4,096 x 512 of 8 1,129 and 609.
inline bool wide_back(const LruGeo& g, int T) {
    const Shape s = shape_of(g, T, kWide, kBackTokens);
    return g.W > 64 && s.segs > 1 && s.tiles >= 2048;
}
// The shape whose workspace a call needs: never less than a smaller call's.
inline Shape back_room(const LruGeo& g, int T) {
    return wide_back(g, T) ? shape_of(g, T, kWide, kBackTokens) : shape_of(g, T, 64, T <= 32 ? 32 : 64);
}
// A wide tile covers as much as a narrow one where the channels fill it, and less of 136
// channels, say: two blocks of 128 for three of 64.  A launch counts 2^32 threads, so the
// largest calls of such widths take the narrow tiles, by which sizes are accepted.
constexpr int64_t kMostTiles = 1ll << 23;   // of 512 threads
inline Shape back_shape(const LruGeo& g, int T) {
    const Shape s = back_room(g, T);
    return s.tiles < kMostTiles ? s : shape_of(g, T, 64, T <= 32 ? 32 : 64);
}

// The workspace of a chained call: 256 bytes with the counter, then a word of 8
// bytes per channel and tile.
inline size_t chain_bytes(const Shape& s) {
    return s.segs == 1 ? 0 : 256 + static_cast<size_t>(s.tiles) * s.channels * sizeof(uint64_t);
}

static hipError_t clear_chain(void* ws, const Shape& sh, Chain& ch, hipStream_t s) {
    char* p = static_cast<char*>(ws);
    ch.next = reinterpret_cast<unsigned*>(p);
    ch.words = reinterpret_cast<uint64_t*>(p + 256);
    const int64_t words = sh.tiles * sh.channels / 2;   // of 16 bytes
    const int64_t grid = (words + 1023) / 1024;
    hipLaunchKernelGGL(lru_clear_kernel, dim3(static_cast<unsigned>(grid < 2048 ? grid : 2048)), dim3(256), 0, s,
                       reinterpret_cast<uint4*>(p + 256), words, ch.next);
    return hipGetLastError();
}

template <typename Act, int LPC, int WAVES, int N, bool GATE, bool CHAIN>
static hipError_t scan_launch(const LruGeo& g, const LruArgs& a, int T, const int32_t* lengths, float* saved,
                              int32_t* status, const Shape& sh, const Chain& ch, hipStream_t s) {
    hipLaunchKernelGGL((lru_scan_kernel<Act, LPC, WAVES, N, GATE, CHAIN>), dim3(static_cast<unsigned>(sh.tiles)),
                       dim3(WAVES * kWave), 0, s, a.state, static_cast<const Act*>(a.x), static_cast<const Act*>(a.r),
                       static_cast<const Act*>(a.i), a.A, static_cast<const Act*>(a.z), lengths,
                       static_cast<Act*>(a.y), saved, status, T, g.W, sh.blocks, g.B * sh.blocks, sh.segs, ch, g.p);
    return hipGetLastError();
}

template <typename Act, bool GATE>
static hipError_t scan_cfg(const LruGeo& g, const LruArgs& a, int T, const int32_t* lengths, float* saved,
                           int32_t* status, void* ws, hipStream_t s) {
    const Shape sh = scan_shape(g, T);
    Chain ch = {};
    if (sh.segs > 1) {
        const hipError_t e = clear_chain(ws, sh, ch, s);
        if (e != hipSuccess)
            return e;
        if (sh.channels == kWide)
            return scan_launch<Act, 32, 8, 8, GATE, true>(g, a, T, lengths, saved, status, sh, ch, s);
        return scan_launch<Act, 16, 8, 4, GATE, true>(g, a, T, lengths, saved, status, sh, ch, s);
    }
    switch (sh.tokens) {
        case 32: return scan_launch<Act, 16, 4, 2, GATE, false>(g, a, T, lengths, saved, status, sh, ch, s);
        case 64: return scan_launch<Act, 16, 8, 2, GATE, false>(g, a, T, lengths, saved, status, sh, ch, s);
        case 128: return scan_launch<Act, 16, 8, 4, GATE, false>(g, a, T, lengths, saved, status, sh, ch, s);
        default: return scan_launch<Act, 16, 8, 8, GATE, false>(g, a, T, lengths, saved, status, sh, ch, s);
    }
}

template <typename Act, int LPC, int WAVES, int N, bool GATE, bool CHAIN>
static hipError_t backward_launch(const LruGeo& g, const LruGrads& a, int T, const int32_t* lengths, int32_t* status,
                                  float* parts, const Shape& sh, const Chain& ch, hipStream_t s) {
    hipLaunchKernelGGL((lru_backward_kernel<Act, LPC, WAVES, N, GATE, CHAIN>), dim3(static_cast<unsigned>(sh.tiles)),
                       dim3(WAVES * kWave), 0, s, static_cast<const Act*>(a.x), static_cast<const Act*>(a.r),
                       static_cast<const Act*>(a.i), a.A, static_cast<const Act*>(a.z), lengths, a.saved,
                       static_cast<const Act*>(a.dy), a.dstate, static_cast<Act*>(a.dx), static_cast<Act*>(a.dr),
                       static_cast<Act*>(a.di), static_cast<Act*>(a.dz), a.dstate0, parts, status, T, g.W, sh.blocks,
                       g.B * sh.blocks, sh.segs, ch, g.p, g.gp);
    return hipGetLastError();
}

inline size_t parts_bytes(const LruGeo& g, const Shape& sh) {
    return (static_cast<size_t>(g.B) * sh.segs * g.W * sizeof(float) + 255) / 256 * 256;
}

template <typename Act, bool GATE>
static hipError_t backward_cfg(const LruGeo& g, const LruGrads& a, int T, const int32_t* lengths, int32_t* status,
                               void* ws, hipStream_t s) {
    const Shape sh = back_shape(g, T);
    float* parts = static_cast<float*>(ws);
    Chain ch = {};
    hipError_t e = hipSuccess;
    if (sh.segs > 1)
        e = clear_chain(static_cast<char*>(ws) + parts_bytes(g, sh), sh, ch, s);
    if (e != hipSuccess)
        return e;
    if (sh.channels == kWide)
        e = backward_launch<Act, 32, 8, 2, GATE, true>(g, a, T, lengths, status, parts, sh, ch, s);
    else if (sh.segs > 1)
        e = backward_launch<Act, 16, 8, 2, GATE, true>(g, a, T, lengths, status, parts, sh, ch, s);
    else if (sh.tokens == 64)
        e = backward_launch<Act, 16, 8, 2, GATE, false>(g, a, T, lengths, status, parts, sh, ch, s);
    else
        e = backward_launch<Act, 16, 4, 2, GATE, false>(g, a, T, lengths, status, parts, sh, ch, s);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(lru_rate_kernel, dim3((g.W + 63) / 64), dim3(1024), 0, s, parts, a.A, a.dA, g.B * sh.segs, g.W);
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

size_t lru_prefill_ws_bytes(const LruGeo& g, int T) { return lru::chain_bytes(lru::scan_shape(g, T)); }

hipError_t launch_lru_prefill(const LruGeo& g, const LruArgs& a, int T, const int32_t* lengths, float* saved,
                              int32_t* status, void* ws, hipStream_t s) {
    if (g.bf16)
        return a.z ? lru::scan_cfg<uint16_t, true>(g, a, T, lengths, saved, status, ws, s)
                   : lru::scan_cfg<uint16_t, false>(g, a, T, lengths, saved, status, ws, s);
    return a.z ? lru::scan_cfg<float, true>(g, a, T, lengths, saved, status, ws, s)
               : lru::scan_cfg<float, false>(g, a, T, lengths, saved, status, ws, s);
}

size_t lru_backward_ws_bytes(const LruGeo& g, int T) {
    const lru::Shape sh = lru::back_room(g, T);
    return lru::parts_bytes(g, sh) + lru::chain_bytes(sh);
}

hipError_t launch_lru_backward(const LruGeo& g, const LruGrads& a, int T, const int32_t* lengths, int32_t* status,
                               void* ws, hipStream_t s) {
    if (g.bf16)
        return a.z ? lru::backward_cfg<uint16_t, true>(g, a, T, lengths, status, ws, s)
                   : lru::backward_cfg<uint16_t, false>(g, a, T, lengths, status, ws, s);
    return a.z ? lru::backward_cfg<float, true>(g, a, T, lengths, status, ws, s)
               : lru::backward_cfg<float, false>(g, a, T, lengths, status, ws, s);
}

}  // namespace gdn
