// The selective state space scan, token by token:
//   dt = softplus(dt_raw + dt_bias),  S <- 2^(-e^A_log log2(e) dt) S + dt x b^T
//   out = (S c + D x) silu(z)
// with one [P, N] state per (sequence, head): a batch of few tokens a row.
//
// For a few tokens the state is everything: 8 N P bytes (fp32, in and out)
// against some 6 P a token, so the kernel keeps it in registers and asks for
// all of it at once.  A workgroup owns up to 64 rows p of one head; the N
// columns of a row lie over N / E lanes, E consecutive-by-four elements each,
// so a row loads and stores as whole lines and the sum over n finishes with
// lane exchanges.  All arithmetic is fp32.
//
// With several tokens it is the latency of their inputs that counts, not their
// bytes: a token's are asked for while the one before is computed, and each
// lane finishes one row.  64 rows, 32 heads of 64 x 128, fp32 states: one token
// 22 us (5.9 TB/s), 8 tokens 41 us; with inputs loaded where they are used, one
// element at a time, and one lane finishing all rows, 25 and 56 us.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 256;

template <int N, int ROWS>
__global__ __launch_bounds__(kThreads) void ssm_recurrent_kernel(SsmParams p)
{
    constexpr int LPR = N >= 64 ? 16 : 8;             // lanes a row
    constexpr int E4 = N / LPR / 4;                   // four-element pieces a lane holds of a row
    constexpr int PASS = kThreads / LPR;              // rows the workgroup covers at once
    constexpr int R = ROWS / PASS;                    // rows a thread holds
    static_assert(ROWS % PASS == 0 && (R & (R - 1)) == 0 && R <= LPR, "whole passes of rows, a lane for each");
    const int tid = threadIdx.x, l = tid % LPR, r0 = tid / LPR;
    const int64_t pblocks = p.P / ROWS;
    const int64_t chain = blockIdx.x / pblocks, pb = blockIdx.x - chain * pblocks;
    const int64_t n = chain / p.H, h = chain - n * p.H;
    const int64_t g = h / (p.H / p.G);

    const int64_t slab = (chain * p.P + pb * ROWS + r0) * N + 4 * l;
    float s[R][E4][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < E4; ++i) {
            const int64_t at = slab + static_cast<int64_t>(r) * PASS * N + 4 * LPR * i;
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

    const float rate = -expf(p.A_log[h]) * kLog2eF;
    const float dt_bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = p.D ? p.D[h] : 0.0f;
    // After the sum every lane of a row has it: lane r of them finishes row r.
    const int mine = (l & (R - 1)) * PASS;
    const uint16_t *xs = p.x + n * p.xb + h * p.P + pb * ROWS + r0;
    const uint16_t *zs = p.z ? p.z + n * p.zb + h * p.P + pb * ROWS + r0 + mine : nullptr;
    const uint16_t *bs = p.b + n * p.bb + g * N + 4 * l, *cs = p.c + n * p.cb + g * N + 4 * l;
    const uint16_t *ds = p.dt + n * p.db + h;
    uint16_t *os = p.out + (n * p.seqs.T * p.H + h) * p.P + pb * ROWS + r0 + mine;
    u32x2_t nb[E4], nc[E4];  // the next token's inputs
    uint32_t nx[R], nz = 0, nd = 0;
    const auto load = [&](int64_t t) {
        nd = ds[t * p.dtt];
#pragma unroll
        for (int i = 0; i < E4; ++i) {
            nb[i] = *reinterpret_cast<const u32x2_a2 *>(bs + t * p.bt + 4 * LPR * i);
            nc[i] = *reinterpret_cast<const u32x2_a2 *>(cs + t * p.ct + 4 * LPR * i);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) nx[r] = xs[t * p.xt + r * PASS];
        if (zs)
            nz = zs[t * p.zt];
    };
    if (p.seqs.T > 0)
        load(0);
    for (int64_t t = 0; t < p.seqs.T; ++t) {
        const float raw = lo_f32(nd) + dt_bias;
        const float dt = softplus_f32(raw, dt_plain_above(p.softplus));
        const float keep = exp2_f32(rate * dt);
        float b[E4][4], c[E4][4], x[R];
        const float z = lo_f32(nz);
#pragma unroll
        for (int i = 0; i < E4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                b[i][2 * e] = lo_f32(nb[i][e]);
                b[i][2 * e + 1] = hi_f32(nb[i][e]);
                c[i][2 * e] = lo_f32(nc[i][e]);
                c[i][2 * e + 1] = hi_f32(nc[i][e]);
            }
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = lo_f32(nx[r]);
        if (t + 1 < p.seqs.T)
            load(t + 1);
        float y_mine = 0.0f, x_mine = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float dx = dt * x[r];
            float y = 0.0f;
#pragma unroll
            for (int i = 0; i < E4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[r][i][e] = fmaf(keep, s[r][i][e], dx * b[i][e]);
                    y = fmaf(s[r][i][e], c[i][e], y);
                }
            y = lane_sum<LPR>(y);
            y_mine = (l & (R - 1)) == r ? y : y_mine;
            x_mine = (l & (R - 1)) == r ? x[r] : x_mine;
        }
        if (l < R) {
            float y = fmaf(skip, x_mine, y_mine);
            if (zs)
                y *= silu_f32(z);
            os[t * p.H * p.P] = f32_to_bf16_rne(y);
        }
    }

    if (!p.final_state)
        return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < E4; ++i) {
            const int64_t at = slab + static_cast<int64_t>(r) * PASS * N + 4 * LPR * i;
            if (p.final_kind == kFp32)
                *reinterpret_cast<f32x4_t *>(static_cast<float *>(p.final_state) + at) =
                    f32x4_t{s[r][i][0], s[r][i][1], s[r][i][2], s[r][i][3]};
            else
                *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(p.final_state) + at) =
                    u32x2_t{pack_bf16x2(s[r][i][0], s[r][i][1]), pack_bf16x2(s[r][i][2], s[r][i][3])};
        }
}

template <int N>
hipError_t launch(const SsmParams &p, hipStream_t stream)
{
    const int64_t rows = p.P % 64 == 0 ? 64 : 32, blocks = p.seqs.N * p.H * (p.P / rows);
    if (!grid_fits(blocks, kThreads))
        return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (rows == 64)
        ssm_recurrent_kernel<N, 64><<<grid, dim3(kThreads), 0, stream>>>(p);
    else
        ssm_recurrent_kernel<N, 32><<<grid, dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_recurrent(const SsmParams &p, hipStream_t stream)
{
    switch (p.N) {
    case 32: return launch<32>(p, stream);
    case 64: return launch<64>(p, stream);
    case 128: return launch<128>(p, stream);
    case 256: return launch<256>(p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace layer
}  // namespace kda
