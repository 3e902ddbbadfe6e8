// Norm and position rotation of query and key heads, out to tensors
// (qk_norm_rotary) or, for keys and with the values beside them, into the slots
// of a paged cache (append_kv).  Per head of D channels:
//   y = x / sqrt(mean x^2 + eps) * weight
//   out_i = scale (y_i cos a - y_j sin a),  out_j = scale (y_j cos a + y_i sin a)
// for the R / 2 pairs (i, j) of the first R channels, a = position * inv_freq.
//
// A few operations a cell against 4 bytes: memory bounds it, and for one token a
// request the latency of one load and one store.  An item is two units of VEC
// adjacent channels that are turned together: units l and l + R / (2 VEC) of
// the halves, or, interleaved or behind R, units 2 l and 2 l + 1.  Either way
// an item's frequencies are VEC l on, so a lane holds both ends of its pairs
// and nothing is exchanged.  VEC is 4 where D and R allow it (multiples of 8),
// else 2 (of 4), else 1.  LPR lanes share a row; a workgroup takes the rows of
// as many tokens as fill its lanes once, and works out their angles once, in
// LDS: in turns, with the product and its reduction to half a turn in 64 bits,
// since fp32 has no digits left for a turn's fraction at far positions.
#include <type_traits>

#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load_unit(const uint16_t *p, float f[4], std::integral_constant<int, 4>)
{
    const u32x2_t u = *reinterpret_cast<const u32x2_a2 *>(p);
    f[0] = lo_f32(u[0]);
    f[1] = hi_f32(u[0]);
    f[2] = lo_f32(u[1]);
    f[3] = hi_f32(u[1]);
}
typedef uint32_t u32_a2 __attribute__((aligned(2)));
__device__ __forceinline__ void load_unit(const uint16_t *p, float f[2], std::integral_constant<int, 2>)
{
    const uint32_t u = *reinterpret_cast<const u32_a2 *>(p);
    f[0] = lo_f32(u);
    f[1] = hi_f32(u);
}
__device__ __forceinline__ void load_unit(const uint16_t *p, float f[1], std::integral_constant<int, 1>)
{
    f[0] = bf16_to_f32(*p);
}
template <int VEC>
__device__ __forceinline__ void store_unit(uint16_t *p, const float f[VEC])
{
    if constexpr (VEC == 4)
        *reinterpret_cast<u32x2_a2 *>(p) = u32x2_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
    else if constexpr (VEC == 2)
        *reinterpret_cast<u32_a2 *>(p) = pack_bf16x2(f[0], f[1]);
    else
        *p = f32_to_bf16_rne(f[0]);
}

// LPR lanes of ITEMS items share a row of at most 2 VEC LPR ITEMS channels.
template <int VEC, int LPR, int ITEMS, bool APPEND>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryParams p, int per_wg)
{
    constexpr std::integral_constant<int, VEC> width;
    // a workgroup's tokens times R / 2 angles: at most 256 / LPR tokens, VEC LPR ITEMS angles each
    constexpr int kAngles = kThreads * VEC * ITEMS;
    __shared__ float2 turn[kAngles];
    __shared__ int64_t place[APPEND ? kThreads : 1][2];
    const int tid = threadIdx.x, l = tid % LPR, group = tid / LPR;
    const int64_t tokens = p.B * p.T, first = static_cast<int64_t>(blockIdx.x) * per_wg;
    const int here = static_cast<int>(tokens - first < per_wg ? tokens - first : per_wg);
    const int half = p.positions ? p.R / 2 : 0;

    for (int i = tid; i < here * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const double turns = static_cast<double>(p.positions[first + t]) * static_cast<double>(p.inv_freq[f]) * 0.15915494309189533577;
        const float part = static_cast<float>(2.0 * (turns - rint(turns)));
        float sn, cs;
        sincospif(part, &sn, &cs);
        turn[i] = make_float2(cs * p.scale, sn * p.scale);
    }
    if constexpr (APPEND) {
        if (tid < here) {
            const int64_t slot = p.slots[first + tid];
            const bool in = slot >= 0 && slot < p.slot_count;
            const int64_t page = in ? slot / p.page_size : 0, at = in ? slot - page * p.page_size : 0;
            place[tid][0] = in ? page * p.xc.page + at * p.xc.token : -1;
            place[tid][1] = page * p.yc.page + at * p.yc.token;
        }
    }
    __syncthreads();

    const int rows = p.first + p.second;
    for (int w = group; w < here * rows; w += kThreads / LPR) {
        const int t = w / rows, r = w - t * rows;
        const bool second = r >= p.first;
        const int head = second ? r - p.first : r;
        const int64_t token = first + t, b = token / p.T, at = token - b * p.T;
        const uint16_t *x = (second ? p.y + b * p.yb + at * p.yt : p.x + b * p.xb + at * p.xt) + static_cast<int64_t>(head) * p.D;
        uint16_t *out;
        bool plain = false;  // the values of an append
        if constexpr (APPEND) {
            if (place[t][0] < 0)
                continue;
            out = second ? p.y_out + place[t][1] + head * p.yc.head : p.x_out + place[t][0] + head * p.xc.head;
            plain = second;
        } else {
            out = second ? p.y_out + (token * p.second + head) * p.D : p.x_out + (token * p.first + head) * p.D;
        }

        float a[ITEMS][VEC], c[ITEMS][VEC];
        int ua[ITEMS], uc[ITEMS];  // first channels of an item's units
        bool turned[ITEMS], in[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int item = l + LPR * i;
            in[i] = 2 * VEC * item < p.D;
            turned[i] = VEC * item < half && !plain;
            const bool split = turned[i] && !p.interleaved;
            ua[i] = split ? VEC * item : 2 * VEC * item;
            uc[i] = ua[i] + (split ? half : VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e) a[i][e] = c[i][e] = 0.0f;
            if (in[i]) {
                load_unit(x + ua[i], a[i], width);
                load_unit(x + uc[i], c[i], width);
            }
        }
        const void *weight = second ? p.y_weight : p.x_weight;
        if (weight && !plain) {
            const int kind = second ? p.y_kind : p.x_kind;
            float wa[ITEMS][VEC], wc[ITEMS][VEC];
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (in[i]) {
                    if (kind == kBf16) {
                        load_unit(static_cast<const uint16_t *>(weight) + ua[i], wa[i], width);
                        load_unit(static_cast<const uint16_t *>(weight) + uc[i], wc[i], width);
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            wa[i][e] = static_cast<const float *>(weight)[ua[i] + e];
                            wc[i][e] = static_cast<const float *>(weight)[uc[i] + e];
                        }
                    }
                }
            const auto squares = [&] {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss = fmaf(a[i][e], a[i][e], fmaf(c[i][e], c[i][e], ss));
                return lane_sum<LPR>(ss) / static_cast<float>(p.D);
            };
            float m = squares() + p.eps.plain;
            if (!norm_in_range(m)) {  // one row's lanes together: m is theirs
                const float f = norm_shift(m), eps = shifted_eps(p.eps, m);
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        a[i][e] *= f;
                        c[i][e] *= f;
                    }
                m = squares() + eps;
            }
            const float s = __builtin_amdgcn_rsqf(m);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (in[i]) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        a[i][e] *= s * wa[i][e];
                        c[i][e] *= s * wc[i][e];
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (!in[i])
                continue;
            if (turned[i]) {
                float v[2 * VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[e] = a[i][e];
                    v[VEC + e] = c[i][e];
                }
                const float2 *cs = turn + t * half + VEC * (l + LPR * i);
                float o[2 * VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 f = cs[e];
                    if (p.interleaved) {
                        o[2 * e] = fmaf(v[2 * e], f.x, -(v[2 * e + 1] * f.y));
                        o[2 * e + 1] = fmaf(v[2 * e + 1], f.x, v[2 * e] * f.y);
                    } else {
                        o[e] = fmaf(v[e], f.x, -(v[VEC + e] * f.y));
                        o[VEC + e] = fmaf(v[VEC + e], f.x, v[e] * f.y);
                    }
                }
                store_unit<VEC>(out + ua[i], o);
                store_unit<VEC>(out + uc[i], o + VEC);
            } else {
                store_unit<VEC>(out + ua[i], a[i]);
                store_unit<VEC>(out + uc[i], c[i]);
            }
        }
    }
}

template <int VEC, int LPR, int ITEMS>
hipError_t launch(const RotaryParams &p, hipStream_t stream)
{
    const int64_t rows = p.first + p.second, fill = kThreads / LPR;
    const int per_wg = static_cast<int>(rows >= fill ? 1 : fill / rows);
    const int64_t blocks = (p.B * p.T + per_wg - 1) / per_wg;
    if (!grid_fits(blocks, kThreads))
        return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (p.slots)
        rotary_kernel<VEC, LPR, ITEMS, true><<<grid, dim3(kThreads), 0, stream>>>(p, per_wg);
    else
        rotary_kernel<VEC, LPR, ITEMS, false><<<grid, dim3(kThreads), 0, stream>>>(p, per_wg);
    return hipGetLastError();
}

// The fewest lanes that hold a row, at most a wave.
template <int VEC>
hipError_t by_size(const RotaryParams &p, hipStream_t stream)
{
    const int items = p.D / (2 * VEC);
    if (items <= 8) return launch<VEC, 8, 1>(p, stream);
    if (items <= 16) return launch<VEC, 16, 1>(p, stream);
    if (items <= 32) return launch<VEC, 32, 1>(p, stream);
    if (items <= 64) return launch<VEC, 64, 1>(p, stream);
    if constexpr (VEC < 4)
        if (items <= 128) return launch<VEC, 64, 2>(p, stream);
    if constexpr (VEC < 2)
        if (items <= 256) return launch<VEC, 64, 4>(p, stream);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rotary(const RotaryParams &p, hipStream_t stream)
{
    const int sizes = p.positions ? p.D | p.R : p.D;
    if (sizes % 8 == 0) return by_size<4>(p, stream);
    if (sizes % 4 == 0) return by_size<2>(p, stream);
    return by_size<1>(p, stream);
}

}  // namespace layer
}  // namespace kda
