// The gated delta rule with one decay per head, token by token:
//   S <- 2^(-e^A_log log2(e) softplus(g + dt_bias)) S
//   u = sigmoid(beta) (v - S k),  S <- S + u k^T,  out = scale S q
// with one [V, K] state per (sequence, head).
//
// For a few tokens the state is everything: 8 K V bytes (fp32, in and out) against
// some 4 (K + V) a token, so it stays in registers and is asked for all at once.
// A workgroup owns up to 64 rows of one head; the K columns of a row lie over 16
// lanes, four adjacent elements at a time, so a row loads and stores as whole
// lines.  Both products of a token, S k and S q, are taken of the state before
// it, one pass over the registers, and joined by
//   scale S' q = scale (decay S q + u (k . q)).
// All arithmetic is fp32.
//
// 64 sequences of one token, 32 heads of 128 x 128, fp32 states: 52 us (5.3 TB/s of
// 272 MB, a large copy's rate) with other states in every call, 43 with the same.  Each
// token more adds 5 to 7 us there; where that passes the chunked kernel's 113 stands
// with the rule of which one runs.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 256, LPR = 16, PASS = kThreads / LPR;  // lanes a row, rows at once

template <int K, int ROWS>
__global__ __launch_bounds__(kThreads) void delta_recurrent_kernel(DeltaParams p)
{
    constexpr int E4 = K / LPR / 4;  // four-element pieces a lane holds of a row
    constexpr int R = ROWS / PASS;   // rows a thread holds
    const int tid = threadIdx.x, l = tid % LPR, r0 = tid / LPR;
    const int64_t vblocks = p.V / ROWS;
    const int64_t chain = blockIdx.x / vblocks, vb = blockIdx.x - chain * vblocks;
    const int64_t n = chain / p.H, h = chain - n * p.H;
    const int64_t grp = h / (p.H / p.G);
    int64_t row = n, begin = 0, end = p.seqs.T;
    if (p.seqs.cu) {
        row = 0;
        begin = clamp_offset(p.seqs, n);
        end = clamp_offset(p.seqs, n + 1);
    }

    const int64_t slab = (chain * p.V + vb * ROWS + r0) * K + 4 * l;
    float s[R][E4][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < E4; ++i) {
            const int64_t at = slab + static_cast<int64_t>(r) * PASS * K + 4 * LPR * i;
            if (p.init_kind == kFp32) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p.init_state) + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[r][i][e] = v[e];
            } else if (p.init_kind == kBf16) {
                const u32x2_t v = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(p.init_state) + at);
                s[r][i][0] = lo_f32(v[0]);
                s[r][i][1] = hi_f32(v[0]);
                s[r][i][2] = lo_f32(v[1]);
                s[r][i][3] = hi_f32(v[1]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[r][i][e] = 0.0f;
            }
        }

    const float rate = -expf(p.A_log[h]) * kLog2eF, bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    // After the sums every lane of a row has them: lane r finishes row r.
    const int mine = (l & (R - 1)) * PASS;
    const int64_t v0 = h * p.V + vb * ROWS + r0;
    const uint16_t *vs = p.v + row * p.vb + v0, *gs = p.g + row * p.gb + h, *bs = p.beta + row * p.bb + h;
    const uint16_t *ks = p.k + row * p.kb + grp * K + 4 * l, *qs = p.q + row * p.qb + grp * K + 4 * l;
    uint16_t *os = p.out + row * p.seqs.T * p.H * p.V + v0 + mine;
    u32x2_t nk[E4], nq[E4];  // the next token's inputs
    uint32_t nv[R], ng = 0, nb = 0;
    const auto load = [&](int64_t t) {
        ng = gs[t * p.gt];
        nb = bs[t * p.bt];
#pragma unroll
        for (int i = 0; i < E4; ++i) {
            nk[i] = *reinterpret_cast<const u32x2_a2 *>(ks + t * p.kt + 4 * LPR * i);
            nq[i] = *reinterpret_cast<const u32x2_a2 *>(qs + t * p.qt + 4 * LPR * i);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) nv[r] = vs[t * p.vt + r * PASS];
    };
    if (begin < end)
        load(begin);
    for (int64_t t = begin; t < end; ++t) {
        const float keep = exp2_f32(rate * softplus_f32(lo_f32(ng) + bias, dt_plain_above(1)));
        const float strength = sigmoid_f32(lo_f32(nb));
        float k[E4][4], q[E4][4], v[R];
        float kq = 0.0f;
#pragma unroll
        for (int i = 0; i < E4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                k[i][2 * e] = lo_f32(nk[i][e]);
                k[i][2 * e + 1] = hi_f32(nk[i][e]);
                q[i][2 * e] = lo_f32(nq[i][e]);
                q[i][2 * e + 1] = hi_f32(nq[i][e]);
            }
#pragma unroll
        for (int i = 0; i < E4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) kq = fmaf(k[i][e], q[i][e], kq);
        kq = lane_sum<LPR>(kq);
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = lo_f32(nv[r]);
        if (t + 1 < end)
            load(t + 1);
        float y_mine = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float sk = 0.0f, sq = 0.0f;
#pragma unroll
            for (int i = 0; i < E4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[r][i][e] *= keep;
                    sk = fmaf(s[r][i][e], k[i][e], sk);
                    sq = fmaf(s[r][i][e], q[i][e], sq);
                }
            sk = lane_sum<LPR>(sk);
            sq = lane_sum<LPR>(sq);
            const float u = strength * (v[r] - sk);
#pragma unroll
            for (int i = 0; i < E4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[r][i][e] = fmaf(u, k[i][e], s[r][i][e]);
            const float y = fmaf(u, kq, sq);
            y_mine = (l & (R - 1)) == r ? y : y_mine;
        }
        if (l < R)
            os[t * p.H * p.V] = f32_to_bf16_rne(p.scale * y_mine);
    }

    if (!p.final_state)
        return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < E4; ++i) {
            const int64_t at = slab + static_cast<int64_t>(r) * PASS * K + 4 * LPR * i;
            if (p.final_kind == kFp32)
                *reinterpret_cast<f32x4_t *>(static_cast<float *>(p.final_state) + at) =
                    f32x4_t{s[r][i][0], s[r][i][1], s[r][i][2], s[r][i][3]};
            else
                *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(p.final_state) + at) =
                    u32x2_t{pack_bf16x2(s[r][i][0], s[r][i][1]), pack_bf16x2(s[r][i][2], s[r][i][3])};
        }
}

template <int K>
hipError_t launch(const DeltaParams &p, hipStream_t stream)
{
    const int64_t rows = p.V % 64 == 0 ? 64 : p.V % 32 == 0 ? 32 : 16, blocks = p.seqs.N * p.H * (p.V / rows);
    if (!grid_fits(blocks, kThreads))
        return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (rows == 64)
        delta_recurrent_kernel<K, 64><<<grid, dim3(kThreads), 0, stream>>>(p);
    else if (rows == 32)
        delta_recurrent_kernel<K, 32><<<grid, dim3(kThreads), 0, stream>>>(p);
    else
        delta_recurrent_kernel<K, 16><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_recurrent(const DeltaParams &p, hipStream_t stream)
{
    switch (p.K) {
    case 64: return launch<64>(p, stream);
    case 128: return launch<128>(p, stream);
    case 256: return launch<256>(p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace layer
}  // namespace kda
