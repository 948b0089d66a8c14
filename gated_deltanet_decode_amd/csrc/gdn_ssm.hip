// gdn_ssm.hip -- the selective state space layer token by token: one decoded
// token in one launch, and the token walk over a prompt.
//
// Decode moves the state once in and once out, 8*H*P*N bytes per sequence
// against 6 flops per state entry: HBM sets the time once there are enough
// sequences (64 of 48 heads of 128 x 128: 416 MB in 67.6 us, 6.2 TB/s), the launch
// itself before that (one: 4.8 us).  The layout is the delta-rule token
// kernel's: a row of N entries over 16 (N = 32: 8) lanes, so that the read-out
// S C is a short DPP sum, with the few conv loads issued ahead of the state
// loads because the memory counter retires in order.  Every workgroup convolves
// the B and C channels of its group itself (2N of them, two per thread at
// N = 256); the tail goes to a second buffer so that no reader of a shared
// channel's window races its writer.
#include "gdn.h"
#include "gdn_ssm.hpp"

namespace gdn {
namespace ssm {

template <int N, int PASSES, typename Act>
__global__ __launch_bounds__(256) void ssm_token_kernel(float* __restrict__ S, const Act* __restrict__ tail_in,
                                                        Act* __restrict__ tail_out, const Act* __restrict__ w,
                                                        const Act* __restrict__ bias, const Act* __restrict__ x,
                                                        const float* __restrict__ dt, const float* __restrict__ dt_bias,
                                                        const float* __restrict__ A, const float* __restrict__ Dskip,
                                                        const Act* __restrict__ z, Act* __restrict__ y, int H, int G,
                                                        int P, int C, int blocks_per_head) {
    using R = Rows<N>;
    using Q = Quad<Act>;
    constexpr int NV = R::NV, LPR = R::LPR;
    constexpr int ROWS_WG = R::PASS * PASSES;
    constexpr int NCH = 2 * N + ROWS_WG;
    constexpr int SLOTS = (NCH + 255) / 256;

    const int blk = blockIdx.x % blocks_per_head;
    const int bh = blockIdx.x / blocks_per_head;
    const int h = bh % H;
    const int seq = bh / H;
    const int rep = H / G;
    const int grp = h / rep;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = tid / kWave;
    const int r = lane % LPR;
    const int row_base = blk * ROWS_WG;
    const bool bc_writer = (h % rep == 0) && blk == 0;

    const size_t seq_c = static_cast<size_t>(seq) * C;
    int chan[SLOTS];
    typename Q::raw traw[SLOTS], wraw[SLOTS];
    Act xin[SLOTS], braw[SLOTS];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
        const int ch0 = tid + 256 * k;
        const int ch = ch0 < NCH ? ch0 : NCH - 1;   // clamped: loads stay unconditional
        chan[k] = ch < N ? H * P + grp * N + ch
                : ch < 2 * N ? H * P + G * N + grp * N + (ch - N)
                             : h * P + row_base + (ch - 2 * N);
        traw[k] = Q::load(tail_in + (seq_c + chan[k]) * 4);
        xin[k] = x[seq_c + chan[k]];
        wraw[k] = Q::load(w + static_cast<size_t>(chan[k]) * 4);
        braw[k] = bias ? bias[chan[k]] : Act(0);
    }
    const float dt_raw = dt[bh] + (dt_bias ? dt_bias[h] : 0.0f);
    const float rate = rate2(A[h]);
    const float skip = Dskip ? Dskip[h] : 0.0f;

    float* Sh = S + static_cast<size_t>(bh) * P * N;
    int row[PASSES];
    float4 s[PASSES][NV];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        row[p] = row_base + p * R::PASS + wave * R::RPW + lane / LPR;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            s[p][j] = load_stream(Sh + row[p] * N + R::key(j, r));
    }

    __shared__ __align__(16) float us[NCH];   // B | C | x rows
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
        const int ch0 = tid + 256 * k;
        const typename Q::raw t = Q::push(traw[k], xin[k]);
        if (ch0 < NCH && (ch0 >= 2 * N || bc_writer))
            Q::store(tail_out + (seq_c + chan[k]) * 4, t);
        float win[4], wf[4];
        Q::to_float(t, win);
        Q::to_float(wraw[k], wf);
        if (ch0 < NCH)
            us[ch0] = conv_bias_silu(wf, win, widen(braw[k]));
    }
    const float step = step_size(dt_raw);
    const float decay = __builtin_amdgcn_exp2f(step * rate);
    __syncthreads();

    float4 bb[NV], cc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        bb[j] = *reinterpret_cast<const float4*>(us + R::key(j, r));
        cc[j] = *reinterpret_cast<const float4*>(us + N + R::key(j, r));
    }
    const size_t yo = static_cast<size_t>(bh) * P;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const float xv = us[2 * N + row[p] - row_base];
        const float u = step * xv;
        float acc = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            s[p][j] = axpby4(u, bb[j], decay, s[p][j]);
            acc = dot4(s[p][j], cc[j], acc);
            store_stream(Sh + row[p] * N + R::key(j, r), s[p][j]);
        }
        acc = group_sum<LPR>(acc);
        if (r == 0) {
            float out = __builtin_fmaf(skip, xv, acc);
            if (z)
                out *= silu(widen(z[yo + row[p]]));
            narrow(out, y[yo + row[p]]);
        }
    }
}

template <int N, int PASSES, typename Act>
static hipError_t token_cfg(const SsmGeo& g, const SsmArgs& a, hipStream_t s) {
    const int bph = g.P / (Rows<N>::PASS * PASSES);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(g.B) * g.H * bph)), block(256);
    hipLaunchKernelGGL((ssm_token_kernel<N, PASSES, Act>), grid, block, 0, s, a.state,
                       static_cast<const Act*>(a.tail_in), static_cast<Act*>(a.tail_out),
                       static_cast<const Act*>(a.w), static_cast<const Act*>(a.bias), static_cast<const Act*>(a.x),
                       a.dt, a.dt_bias, a.A, a.D, static_cast<const Act*>(a.z), static_cast<Act*>(a.y), g.H, g.G, g.P,
                       g.C, bph);
    return hipGetLastError();
}

template <typename Act>
static hipError_t token_act(const SsmGeo& g, const SsmArgs& a, hipStream_t s) {
    // Once there are enough (sequence, head) pairs to fill the chip, more rows per
    // workgroup share its conv.  Calls back to back at batch 64: N = 64 (64 heads of 64
    // rows) 37.4 us with 16 rows, 28.7 with 32, 26.3 with 64; N = 128 (48 heads of 128
    // rows) 79, 69.7 and 71.1 us.  Few pairs want many workgroups instead.
    const bool many = static_cast<int64_t>(g.B) * g.H >= 512;
    switch (g.N) {
        case 32: return token_cfg<32, 1, Act>(g, a, s);
        case 64:
            return !many       ? token_cfg<64, 1, Act>(g, a, s)
                   : g.P == 32 ? token_cfg<64, 2, Act>(g, a, s)
                               : token_cfg<64, 4, Act>(g, a, s);
        case 128: return many ? token_cfg<128, 2, Act>(g, a, s) : token_cfg<128, 1, Act>(g, a, s);
        default: return token_cfg<256, 1, Act>(g, a, s);
    }
}

// The token walk: one workgroup per (sequence, head, PASS state rows) holds its
// rows in registers and steps through the sequence's tokens, with the next
// token's inputs loaded one step ahead and one barrier per token.
template <int N, typename Act>
__global__ __launch_bounds__(256) void ssm_walk_kernel(float* __restrict__ S, const Act* __restrict__ tail,
                                                       const Act* __restrict__ w, const Act* __restrict__ bias,
                                                       const Act* __restrict__ x, const float* __restrict__ dt,
                                                       const float* __restrict__ dt_bias, const float* __restrict__ A,
                                                       const float* __restrict__ Dskip, const Act* __restrict__ z,
                                                       Act* __restrict__ y, const int32_t* __restrict__ lengths, int T,
                                                       int H, int G, int P, int C, int blocks_per_head) {
    using R = Rows<N>;
    using Q = Quad<Act>;
    constexpr int NV = R::NV, LPR = R::LPR;
    constexpr int NCH = 2 * N + R::PASS;
    constexpr int SLOTS = (NCH + 255) / 256;

    const int blk = blockIdx.x % blocks_per_head;
    const int bh = blockIdx.x / blocks_per_head;
    const int h = bh % H;
    const int seq = bh / H;
    const int grp = h / (H / G);
    const int len = lengths ? lengths[seq] : T;
    if (len < 1 || len > T)   // nothing to do, or refused (ssm_tail_kernel reports it)
        return;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = tid / kWave;
    const int r = lane % LPR;
    const int row_base = blk * R::PASS;

    const Act* xs = x + static_cast<size_t>(seq) * T * C;
    const float* dts = dt + static_cast<size_t>(seq) * T * H + h;
    int chan[SLOTS];
    float win[SLOTS][4], wf[SLOTS][4], bf[SLOTS];
    Act xin[SLOTS];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
        const int ch0 = tid + 256 * k;
        const int ch = ch0 < NCH ? ch0 : NCH - 1;
        chan[k] = ch < N ? H * P + grp * N + ch
                : ch < 2 * N ? H * P + G * N + grp * N + (ch - N)
                             : h * P + row_base + (ch - 2 * N);
        Q::to_float(Q::load(tail + (static_cast<size_t>(seq) * C + chan[k]) * 4), win[k]);
        Q::to_float(Q::load(w + static_cast<size_t>(chan[k]) * 4), wf[k]);
        bf[k] = bias ? widen(bias[chan[k]]) : 0.0f;
        xin[k] = xs[chan[k]];
    }
    float dt_in = dts[0];
    const float dtb = dt_bias ? dt_bias[h] : 0.0f;
    const float rate = rate2(A[h]);
    const float skip = Dskip ? Dskip[h] : 0.0f;

    const int row = row_base + wave * R::RPW + lane / LPR;
    float* Sr = S + (static_cast<size_t>(bh) * P + row) * N;
    float4 s[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        s[j] = load_stream(Sr + R::key(j, r));

    __shared__ __align__(16) float us[2][NCH];
    for (int t = 0; t < len; ++t) {
        float* u = us[t & 1];
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            win[k][0] = win[k][1];
            win[k][1] = win[k][2];
            win[k][2] = win[k][3];
            win[k][3] = widen(xin[k]);
            const float v = conv_bias_silu(wf[k], win[k], bf[k]);
            if (tid + 256 * k < NCH)
                u[tid + 256 * k] = v;
        }
        const float step = step_size(dt_in + dtb);
        const float decay = __builtin_amdgcn_exp2f(step * rate);
        if (t + 1 < len) {
#pragma unroll
            for (int k = 0; k < SLOTS; ++k)
                xin[k] = xs[static_cast<size_t>(t + 1) * C + chan[k]];
            dt_in = dts[static_cast<size_t>(t + 1) * H];
        }
        __syncthreads();   // two buffers: the next token's conv never overwrites what a slower wave still reads
        const float xv = u[2 * N + row - row_base];
        const float ux = step * xv;
        float acc = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            s[j] = axpby4(ux, *reinterpret_cast<const float4*>(u + R::key(j, r)), decay, s[j]);
            acc = dot4(s[j], *reinterpret_cast<const float4*>(u + N + R::key(j, r)), acc);
        }
        acc = group_sum<LPR>(acc);
        if (r == 0) {
            const size_t yo = (static_cast<size_t>(seq) * T + t) * H * P + static_cast<size_t>(h) * P + row;
            float out = __builtin_fmaf(skip, xv, acc);
            if (z)
                out *= silu(widen(z[yo]));
            narrow(out, y[yo]);
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        store_stream(Sr + R::key(j, r), s[j]);
}

// The conv tail after a prompt (the last four raw inputs of tail ++ x), one
// thread per (sequence, channel), and the sequences' status words.  It runs
// after every reader of the old tail.
template <typename Act>
__global__ __launch_bounds__(256) void ssm_tail_kernel(Act* __restrict__ tail, const Act* __restrict__ x,
                                                       const int32_t* __restrict__ lengths,
                                                       int32_t* __restrict__ status, int T, int C) {
    using Q = Quad<Act>;
    const int blocks = (C + 255) / 256;
    const int seq = blockIdx.x / blocks;
    const int c = (blockIdx.x % blocks) * 256 + threadIdx.x;
    const int len = lengths ? lengths[seq] : T;
    const bool bad = len < 0 || len > T;
    if (status && c == 0)
        status[seq] = bad ? GDN_ERR_INDEX : GDN_OK;
    if (bad || len == 0 || c >= C)
        return;
    Act* tp = tail + (static_cast<size_t>(seq) * C + c) * 4;
    typename Q::raw t = Q::load(tp);
    const Act* xs = x + static_cast<size_t>(seq) * T * C + c;
#pragma unroll
    for (int j = 4; j >= 1; --j)
        if (len >= j)
            t = Q::push(t, xs[static_cast<size_t>(len - j) * C]);
    Q::store(tp, t);
}

template <int N, typename Act>
static hipError_t walk_cfg(const SsmGeo& g, const SsmArgs& a, int T, const int32_t* lengths, hipStream_t s) {
    const int bph = g.P / Rows<N>::PASS;
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(g.B) * g.H * bph)), block(256);
    hipLaunchKernelGGL((ssm_walk_kernel<N, Act>), grid, block, 0, s, a.state, static_cast<const Act*>(a.tail_in),
                       static_cast<const Act*>(a.w), static_cast<const Act*>(a.bias), static_cast<const Act*>(a.x),
                       a.dt, a.dt_bias, a.A, a.D, static_cast<const Act*>(a.z), static_cast<Act*>(a.y), lengths, T, g.H,
                       g.G, g.P, g.C, bph);
    return hipGetLastError();
}

template <typename Act>
static hipError_t prefill_act(const SsmGeo& g, const SsmArgs& a, int T, const int32_t* lengths, int32_t* status,
                              void* ws, hipStream_t s) {
    hipError_t e;
    if (T > walk_tokens(g))
        return launch_ssm_chunked(g, a, T, lengths, status, ws, s);
    switch (g.N) {
        case 32: e = walk_cfg<32, Act>(g, a, T, lengths, s); break;
        case 64: e = walk_cfg<64, Act>(g, a, T, lengths, s); break;
        case 128: e = walk_cfg<128, Act>(g, a, T, lengths, s); break;
        default: e = walk_cfg<256, Act>(g, a, T, lengths, s); break;
    }
    if (e != hipSuccess)
        return e;
    const int64_t blocks = (g.C + 255) / 256;
    hipLaunchKernelGGL(ssm_tail_kernel<Act>, dim3(static_cast<unsigned>(g.B * blocks)), dim3(256), 0, s,
                       static_cast<Act*>(a.tail_out), static_cast<const Act*>(a.x), lengths, status, T, g.C);
    return hipGetLastError();
}

}  // namespace ssm

hipError_t launch_ssm_token(const SsmGeo& g, const SsmArgs& a, hipStream_t s) {
    return g.bf16 ? ssm::token_act<uint16_t>(g, a, s) : ssm::token_act<float>(g, a, s);
}

size_t ssm_prefill_ws_bytes(const SsmGeo& g, int T) { return T > ssm::walk_tokens(g) ? ssm::chunked_ws_bytes(g, T) : 256; }

hipError_t launch_ssm_prefill(const SsmGeo& g, const SsmArgs& a, int T, const int32_t* lengths, int32_t* status,
                              void* ws, hipStream_t s) {
    return g.bf16 ? ssm::prefill_act<uint16_t>(g, a, T, lengths, status, ws, s)
                  : ssm::prefill_act<float>(g, a, T, lengths, status, ws, s);
}

}  // namespace gdn
