// The norms around a block, each one pass over its rows.
//
// gated_norm (after a mixer), over groups of `group` channels:
//   out = v / sqrt(mean v^2 + eps) * w * act(gate),  v = x, or
//   out = v / sqrt(mean v^2 + eps) * w,              v = x * act(gate)
// residual_norm (between two blocks), over rows of D channels:
//   y = x, or x / sqrt(mean x^2 + eps) * post_w
//   r = residual_scale * residual + block_scale * gate * y
//   residual_out = r,  out = r / sqrt(mean r^2 + eps) * w
//
// A few operations a cell against 6 to 14 bytes: memory bounds both.  A row
// stays in the registers of the threads that share it (TPR threads, K vectors
// of eight elements each), so every tensor is touched once.  Rows of up to
// 512 elements are shared by 8 to 64 lanes of one wave, and their sums never
// leave it; longer rows by a workgroup of 256, whose four waves meet in LDS.
// Sums and the values between the two norms are fp32; the second norm takes
// the unrounded r.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 256;

// Sum over the TPR threads of a row.  `part` is LDS for TPR > 64; a second
// sum in the same kernel takes another one, so one barrier serves each.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *part)
{
    if constexpr (TPR <= 64) {
        return lane_sum<TPR>(x);
    } else {
        x = lane_sum<64>(x);
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = x;
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) s += part[i];
        return s;
    }
}

__device__ __forceinline__ float inv_rms(float ss, float n, float eps)
{
    return __builtin_amdgcn_rsqf(ss / n + eps);
}

template <int TPR, int K>
__global__ __launch_bounds__(kThreads) void gated_norm_kernel(GatedParams p, int64_t groups, int64_t per_row)
{
    __shared__ float part[kThreads / 64];
    const int r = threadIdx.x / TPR, l = threadIdx.x % TPR;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + r;
    if (g >= groups)
        return;  // whole rows: TPR threads leave together
    const int64_t row = per_row == 1 ? g : g / per_row, c0 = (g - row * per_row) * p.group;

    float v[K][8], a[K][8];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t at = c0 + (k * TPR + l) * 8;
        const int64_t left = c0 + p.group - at;
        const int count = static_cast<int>(left < 0 ? 0 : (left < 8 ? left : 8));
        unpack8(load8_raw(p.x + row * p.xr + at, count), v[k]);
        if (p.gate)
            unpack8(load8_raw(p.gate + row * p.gr + at, count), a[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = !p.gate ? 1.0f : p.act == kActSilu ? silu_f32(a[k][e]) : sigmoid_f32(a[k][e]);
            a[k][e] = f;
            if (p.gate_first)
                v[k][e] *= f;
            ss = fmaf(v[k][e], v[k][e], ss);
        }
    const float s = inv_rms(row_sum<TPR>(ss, part), static_cast<float>(p.group), p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t at = c0 + (k * TPR + l) * 8;
        const int64_t left = c0 + p.group - at;
        const int count = static_cast<int>(left < 0 ? 0 : (left < 8 ? left : 8));
        if (count <= 0)
            continue;
        float w[8], y[8];
        load8(p.weight, p.weight_kind, at, count, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = v[k][e] * s * w[e];
            if (!p.gate_first)
                y[e] *= a[k][e];
        }
        store8_raw(p.out + row * p.D + at, pack8(y), count);
    }
}

template <int TPR, int K>
__global__ __launch_bounds__(kThreads) void residual_norm_kernel(ResidParams p)
{
    __shared__ float part[2][kThreads / 64];
    const int sub = threadIdx.x / TPR, l = threadIdx.x % TPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + sub;
    if (row >= p.rows)
        return;

    float v[K][8], r[K][8];
    int count[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t at = (k * TPR + l) * 8, left = p.D - at;
        count[k] = static_cast<int>(left < 0 ? 0 : (left < 8 ? left : 8));
        unpack8(load8_raw(p.x + row * p.xr + at, count[k]), v[k]);
        if (p.residual) {
            load8(p.residual, p.residual_kind, row * p.D + at, count[k], r[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[k][e] = 0.0f;
        }
    }
    if (p.post_weight) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[k][e], v[k][e], ss);
        const float s = inv_rms(row_sum<TPR>(ss, part[0]), static_cast<float>(p.D), p.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[8];
            load8(p.post_weight, p.post_kind, (k * TPR + l) * 8, count[k], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= s * w[e];
        }
    }
    float ss = 0.0f;
    const int64_t gate_at = p.gate ? (row / p.gate_period) * p.gr : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (p.gate) {
            float a[8];
            load8(p.gate, p.gate_kind, gate_at + (k * TPR + l) * 8, count[k], a);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= a[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[k][e] = fmaf(p.block_scale, v[k][e], p.residual ? p.residual_scale * r[k][e] : 0.0f);
            ss = fmaf(r[k][e], r[k][e], ss);
        }
        if (p.residual_out && count[k] > 0)
            store8(p.residual_out, p.residual_out_kind, row * p.D + (k * TPR + l) * 8, count[k], r[k]);
    }
    if (!p.out)
        return;
    const float s = inv_rms(row_sum<TPR>(ss, part[1]), static_cast<float>(p.D), p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (count[k] <= 0)
            continue;
        float w[8], y[8];
        load8(p.weight, p.weight_kind, (k * TPR + l) * 8, count[k], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = r[k][e] * s * w[e];
        store8_raw(p.out + row * p.D + (k * TPR + l) * 8, pack8(y), count[k]);
    }
}

// Calls f(threads per row, vectors per thread) for rows of `size` elements:
// the fewest lanes that hold the row at eight elements each, then the
// workgroup with 1 to 8 vectors a thread (16384 elements at most).
template <int A, int B>
struct Pair {
    static constexpr int tpr = A, k = B;
};
template <class F>
hipError_t by_size(int64_t size, F f)
{
    if (size <= 64) return f(Pair<8, 1>());
    if (size <= 128) return f(Pair<16, 1>());
    if (size <= 256) return f(Pair<32, 1>());
    if (size <= 512) return f(Pair<64, 1>());
    if (size <= 2048) return f(Pair<256, 1>());
    if (size <= 4096) return f(Pair<256, 2>());
    if (size <= 8192) return f(Pair<256, 4>());
    if (size <= kMaxNormSize) return f(Pair<256, 8>());
    return hipErrorInvalidValue;
}

bool grid(int64_t rows, int tpr, dim3 *g)
{
    const int64_t per = kThreads / tpr, blocks = (rows + per - 1) / per;
    *g = dim3(static_cast<uint32_t>(blocks));
    return blocks <= INT32_MAX;
}

}  // namespace

hipError_t launch_gated_norm(const GatedParams &p, hipStream_t stream)
{
    const int64_t per_row = p.D / p.group, groups = p.rows * per_row;
    return by_size(p.group, [&](auto c) {
        dim3 g;
        if (!grid(groups, c.tpr, &g))
            return hipErrorInvalidConfiguration;
        gated_norm_kernel<c.tpr, c.k><<<g, dim3(kThreads), 0, stream>>>(p, groups, per_row);
        return hipGetLastError();
    });
}

hipError_t launch_residual_norm(const ResidParams &p, hipStream_t stream)
{
    return by_size(p.D, [&](auto c) {
        dim3 g;
        if (!grid(p.rows, c.tpr, &g))
            return hipErrorInvalidConfiguration;
        residual_norm_kernel<c.tpr, c.k><<<g, dim3(kThreads), 0, stream>>>(p);
        return hipGetLastError();
    });
}

}  // namespace layer
}  // namespace kda
