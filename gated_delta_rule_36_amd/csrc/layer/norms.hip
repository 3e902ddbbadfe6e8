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
// leave it; longer ones by a workgroup of two to eight waves, one vector a
// thread up to 4096 elements, which meet in LDS: as many waves as the row fills
// (8192 rows of 5120: 62 us with five waves, 78 with eight; 4096 rows of 2560:
// 15.6 with five, 18.2 with eight).  Sums and the values between
// the two norms are fp32; the second norm takes the unrounded r.
//
// Measured: gated_norm over 4,194,304 rows of 128, 516 us, 6.2 TB/s;
// residual_norm over 32768 rows of 4096 with an fp32 stream, post norm and
// gate, 280 us, 5.8 TB/s (512 threads a row; 294 us with 256 of two vectors
// each), where a 1 GiB copy reaches 5.1 TB/s.  Asking for more waves a SIMD (8,
// by a register limit) lost 2 to 3 %.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

// TPR of rows shared by a workgroup: 2 to 8 waves, as many as the row fills.
constexpr int kWaves = 0, kMaxThreads = 512;
// Threads of a workgroup: one row where its threads are several waves (at
// most), else as many rows as four waves hold.
template <int TPR>
constexpr int kThreads = TPR == kWaves ? kMaxThreads : 256;

// Workgroups come in lines of 2^kLineShift: the rows of a large batch are more
// than one dimension of a grid takes (2^32 threads).
constexpr int kLineShift = 20;
__device__ __forceinline__ int64_t block_index() { return static_cast<int64_t>(blockIdx.y) << kLineShift | blockIdx.x; }

// The row of a thread, and its place among the row's threads.
struct Place {
    int64_t row;
    int lane;
};
template <int TPR>
__device__ __forceinline__ Place place()
{
    const int t = threadIdx.x;
    if constexpr (TPR == kWaves)
        return {block_index(), t};
    else
        return {block_index() * (256 / TPR) + t / TPR, t % TPR};
}

// Sum over the threads of a row.  `part` is LDS for a workgroup's row; a second
// sum in the same kernel takes another one, so one barrier serves each.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *part, int threads)
{
    if constexpr (TPR != kWaves) {
        return lane_sum<TPR>(x);
    } else {
        x = lane_sum<64>(x);
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = x;
        __syncthreads();
        static_assert(kMaxThreads / 64 == 8, "a sum over groups of eight lanes");
        const int wave = threadIdx.x & 7;
        const float s = part[wave];
        return lane_sum<8>(64 * wave < threads ? s : 0.0f);
    }
}

// 1 / sqrt(mean v^2 + eps) over a row of n elements, of which ss is the thread's
// sum of squares; for a row whose squares fp32 does not hold v comes back scaled
// and what is returned with it.
template <int TPR, int K>
__device__ __forceinline__ float inv_rms(float (&v)[K][8], float ss, float *part, int threads, float n, const NormEps &eps)
{
    float m = row_sum<TPR>(ss, part, threads) / n + eps.plain;
    const bool held = norm_in_range(m);
    // a wave's rows together, or the workgroup's one, whose threads all have m
    if (TPR != kWaves ? __any(!held) : !held) {
        const float f = held ? 1.0f : norm_shift(m), e = held ? eps.plain : shifted_eps(eps, m);
        ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[k][i] *= f;
                ss = fmaf(v[k][i], v[k][i], ss);
            }
        if constexpr (TPR == kWaves)
            __syncthreads();  // the first sum has been read
        m = row_sum<TPR>(ss, part, threads) / n + e;
    }
    return __builtin_amdgcn_rsqf(m);
}

// FULL: the row fills its lanes' vectors.
template <int TPR, int K, bool FULL>
__global__ __launch_bounds__(kThreads<TPR>) void gated_norm_kernel(GatedParams p, int64_t groups, uint32_t per_row, int threads)
{
    __shared__ float part[kThreads<TPR> / 64];
    const Place at_row = place<TPR>();
    const int l = at_row.lane, tpr = TPR == kWaves ? threads : TPR;
    const int64_t g = at_row.row;
    if (g >= groups)
        return;  // whole rows: their threads leave together
    const int64_t row = per_row == 1 ? g : g / per_row, c0 = (g - row * per_row) * p.group;
    const uint16_t *x = p.x + row * p.xr + c0, *gate = p.gate ? p.gate + row * p.gr + c0 : nullptr;

    float v[K][8], a[K][8];
    float ss = 0.0f;
    // with several vectors a thread, the row is longer than half of them
    const auto whole = [](int k) { return FULL || 2 * k + 2 <= K; };
    const auto part_of = [&](int k) {
        const int64_t at = (k * tpr + l) * 8;
        return whole(k) ? Eight{at, 0, 8} : eight_of(at, p.group);
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Eight ch = part_of(k);
        unpack8(load8_raw(x, ch), v[k]);
        if (gate)
            unpack8(load8_raw(gate, ch), a[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Eight ch = part_of(k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = !gate ? 1.0f : p.act == kActSilu ? silu_f32(a[k][e]) : sigmoid_f32(a[k][e]);
            a[k][e] = f;
            if (p.gate_first)
                v[k][e] *= f;
        }
        if (!whole(k))
            keep_own(ch, v[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[k][e], v[k][e], ss);
    }
    const float s = inv_rms<TPR>(v, ss, part, threads, static_cast<float>(p.group), p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Eight ch = part_of(k);
        if (!whole(k) && ch.skip >= ch.count)
            continue;
        float w[8], y[8];
        load8(p.weight, p.weight_kind, c0, ch, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = v[k][e] * s * w[e];
            if (!p.gate_first)
                y[e] *= a[k][e];
        }
        store8_raw(p.out + row * p.D + c0, pack8(y), ch);
    }
}

template <int TPR, int K, bool FULL>
__global__ __launch_bounds__(kThreads<TPR>) void residual_norm_kernel(ResidParams p, int threads)
{
    __shared__ float part[2][kThreads<TPR> / 64];
    const Place at_row = place<TPR>();
    const int l = at_row.lane, tpr = TPR == kWaves ? threads : TPR;
    const int64_t row = at_row.row;
    if (row >= p.rows)
        return;
    // with several vectors a thread, the row is longer than half of them
    const auto whole = [](int k) { return FULL || 2 * k + 2 <= K; };
    const auto part_of = [&](int k) {
        const int64_t at = (k * tpr + l) * 8;
        return whole(k) ? Eight{at, 0, 8} : eight_of(at, p.D);
    };

    float v[K][8], r[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Eight ch = part_of(k);
        unpack8(load8_raw(p.x + row * p.xr, ch), v[k]);
        if (p.residual) {
            load8(p.residual, p.residual_kind, row * p.D, ch, r[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[k][e] = 0.0f;
        }
        if (!whole(k))
            keep_own(ch, v[k]);
    }
    if (p.post_weight) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[k][e], v[k][e], ss);
        const float s = inv_rms<TPR>(v, ss, part[0], threads, static_cast<float>(p.D), p.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[8];
            load8(p.post_weight, p.post_kind, 0, part_of(k), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= s * w[e];
        }
    }
    float ss = 0.0f;
    const int64_t gate_at = p.gate ? (row / p.gate_period) * p.gr : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Eight ch = part_of(k);
        if (p.gate) {
            float a[8];
            load8(p.gate, p.gate_kind, gate_at, ch, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= a[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[k][e] = fmaf(p.block_scale, v[k][e], p.residual ? p.residual_scale * r[k][e] : 0.0f);
        }
        if (!whole(k))
            keep_own(ch, r[k]);  // weights and gates there may be anything
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(r[k][e], r[k][e], ss);
        if (p.residual_out && (whole(k) || ch.skip < ch.count))
            store8(p.residual_out, p.residual_out_kind, row * p.D, ch, r[k]);
    }
    if (!p.out)
        return;
    const float s = inv_rms<TPR>(r, ss, part[1], threads, static_cast<float>(p.D), p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Eight ch = part_of(k);
        if (!whole(k) && ch.skip >= ch.count)
            continue;
        float w[8], y[8];
        load8(p.weight, p.weight_kind, 0, ch, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = r[k][e] * s * w[e];
        store8_raw(p.out + row * p.D, pack8(y), ch);
    }
}

// Calls f(threads per row, vectors per thread) for rows of `size` elements:
// the fewest lanes that hold the row at eight elements each, then workgroups of
// as many waves as hold it (16384 elements at most).  With several vectors a
// thread the row is longer than half of them hold.
template <int A, int B, bool C>
struct Shape {
    static constexpr int tpr = A, k = B;
    static constexpr bool full = C;
    int threads;  // of a row
};
template <int A, int B, class F>
hipError_t with_shape(int64_t size, F f)
{
    const int threads = A != kWaves ? A : static_cast<int>((size + 512 * B - 1) / (512 * B) * 64);
    return size == threads * B * 8 ? f(Shape<A, B, true>{threads}) : f(Shape<A, B, false>{threads});
}
template <class F>
hipError_t by_size(int64_t size, F f)
{
    if (size <= 64) return with_shape<8, 1>(size, f);
    if (size <= 128) return with_shape<16, 1>(size, f);
    if (size <= 256) return with_shape<32, 1>(size, f);
    if (size <= 512) return with_shape<64, 1>(size, f);
    if (size <= 4096) return with_shape<kWaves, 1>(size, f);
    if (size <= 8192) return with_shape<kWaves, 2>(size, f);
    if (size <= kMaxNormSize) return with_shape<kWaves, 4>(size, f);
    return hipErrorInvalidValue;
}

bool grid(int64_t rows, int tpr, dim3 *g)
{
    const int64_t per = tpr > 64 ? 1 : 256 / tpr, blocks = (rows + per - 1) / per, line = int64_t(1) << kLineShift;
    if (blocks <= line) {
        *g = dim3(static_cast<uint32_t>(blocks));
        return true;
    }
    const int64_t lines = (blocks + line - 1) / line;
    *g = dim3(static_cast<uint32_t>(line), static_cast<uint32_t>(lines));
    return lines < 65536;
}

}  // namespace

hipError_t launch_gated_norm(const GatedParams &p, hipStream_t stream)
{
    const int64_t per_row = p.D / p.group, groups = p.rows * per_row;
    return by_size(p.group, [&](auto c) {
        dim3 g;
        if (!grid(groups, c.threads, &g))
            return hipErrorInvalidConfiguration;
        gated_norm_kernel<c.tpr, c.k, c.full><<<g, dim3(c.tpr == kWaves ? c.threads : 256), 0, stream>>>(
            p, groups, static_cast<uint32_t>(per_row), c.threads);
        return hipGetLastError();
    });
}

hipError_t launch_residual_norm(const ResidParams &p, hipStream_t stream)
{
    return by_size(p.D, [&](auto c) {
        dim3 g;
        if (!grid(p.rows, c.threads, &g))
            return hipErrorInvalidConfiguration;
        residual_norm_kernel<c.tpr, c.k, c.full><<<g, dim3(c.tpr == kWaves ? c.threads : 256), 0, stream>>>(p, c.threads);
        return hipGetLastError();
    });
}

}  // namespace layer
}  // namespace kda
