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
//
// Beyond kManyBlocks workgroups a lane takes kDepth rows, the next one asked for
// before one is finished, and keeps its weights: 32768 tokens of 40 heads of 128 take
// 137 us (4.9 TB/s; 147 with one or two rows a lane), the append of 19595 tokens of 8
// heads of 128, keys and values, 39 (4.1 TB/s; 57 with one, 43 with two).  Fewer rows go
// one a lane, so that all of the chip has some: 64 tokens take 6 us on the GPU (the
// append 4.5), which is one load, the angles and one store.
#include <algorithm>
#include <type_traits>

#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kManyBlocks = 4096, kDepth = 4;

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
    __shared__ int64_t from[kThreads / LPR][2], to[kThreads / LPR][2];  // where a token's x and y lie, and where they go
    const int tid = threadIdx.x, l = tid % LPR, group = tid / LPR;
    const int64_t tokens = p.B * p.T, first = static_cast<int64_t>(blockIdx.x) * per_wg;
    const int here = static_cast<int>(tokens - first < per_wg ? tokens - first : per_wg);
    const int half = p.positions ? p.R / 2 : 0;

    if (tid < here) {
        const int64_t token = first + tid, b = token / p.T, at = token - b * p.T;
        from[tid][0] = b * p.xb + at * p.xt;
        from[tid][1] = b * p.yb + at * p.yt;
        if constexpr (APPEND) {
            const int64_t slot = p.slots[token];
            const bool in = slot >= 0 && slot < p.slot_count;
            const int64_t page = in ? slot / p.page_size : 0, off = in ? slot - page * p.page_size : 0;
            to[tid][0] = in ? page * p.xc.page + off * p.xc.token : -1;
            to[tid][1] = in ? page * p.yc.page + off * p.yc.token : -1;
        } else {
            to[tid][0] = token * p.first * p.D;
            to[tid][1] = token * p.second * p.D;
        }
    }
    for (int i = tid; i < here * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const double turns = static_cast<double>(p.positions[first + t]) * static_cast<double>(p.inv_freq[f]) * 0.15915494309189533577;
        const float part = static_cast<float>(2.0 * (turns - rint(turns)));
        float sn, cs;
        sincospif(part, &sn, &cs);
        turn[i] = make_float2(cs * p.scale, sn * p.scale);
    }
    __syncthreads();

    const int rows = p.first + p.second;
    const float inverse_size = 1.0f / static_cast<float>(p.D);
    // An item's units start at these channels; the values of an append go as they are.
    const auto turned = [&](bool second, int i) { return VEC * (l + LPR * i) < half && !(APPEND && second); };
    const auto inside = [&](int i) { return 2 * VEC * (l + LPR * i) < p.D; };
    const auto unit_a = [&](bool second, int i) { return (turned(second, i) && !p.interleaved ? VEC : 2 * VEC) * (l + LPR * i); };
    const auto unit_c = [&](bool second, int i) { return unit_a(second, i) + (turned(second, i) && !p.interleaved ? half : VEC); };
    // the weights of x and of y
    float wa[2][ITEMS][VEC], wc[2][ITEMS][VEC];
#pragma unroll
    for (int y = 0; y < (APPEND ? 1 : 2); ++y) {
        const void *weight = y ? p.y_weight : p.x_weight;
        const int kind = y ? p.y_kind : p.x_kind;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (!weight || !inside(i))
                continue;
            const int ua = unit_a(y, i), uc = unit_c(y, i);
            if (kind == kBf16) {
                load_unit(static_cast<const uint16_t *>(weight) + ua, wa[y][i], width);
                load_unit(static_cast<const uint16_t *>(weight) + uc, wc[y][i], width);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    wa[y][i][e] = static_cast<const float *>(weight)[ua + e];
                    wc[y][i][e] = static_cast<const float *>(weight)[uc + e];
                }
            }
        }
    }

    // A row on its way: the next one's numbers are asked for before this one's are used.
    struct Row {
        int t;
        bool second;
        uint16_t *out;  // nullptr: left out
        float a[ITEMS][VEC], c[ITEMS][VEC];
    };
    const auto fetch = [&](int t, int r) {
        Row row;
        row.t = t;
        row.second = r >= p.first;
        const int head = row.second ? r - p.first : r;
        const uint16_t *x = (row.second ? p.y : p.x) + from[t][row.second] + head * p.D;
        const int64_t place = to[t][row.second];
        if constexpr (APPEND)
            row.out = place < 0 ? nullptr : (row.second ? p.y_out : p.x_out) + place + head * (row.second ? p.yc.head : p.xc.head);
        else
            row.out = (row.second ? p.y_out : p.x_out) + place + head * p.D;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) row.a[i][e] = row.c[i][e] = 0.0f;
            if (inside(i)) {
                load_unit(x + unit_a(row.second, i), row.a[i], width);
                load_unit(x + unit_c(row.second, i), row.c[i], width);
            }
        }
        return row;
    };
    const auto finish = [&](Row &row) {
        if ((row.second ? p.y_weight : p.x_weight) && !(APPEND && row.second)) {
            const auto squares = [&] {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss = fmaf(row.a[i][e], row.a[i][e], fmaf(row.c[i][e], row.c[i][e], ss));
                return lane_sum<LPR>(ss) * inverse_size;
            };
            float m = squares() + p.eps.plain;
            if (!norm_in_range(m)) {  // one row's lanes together: m is theirs
                const float f = norm_shift(m), eps = shifted_eps(p.eps, m);
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        row.a[i][e] *= f;
                        row.c[i][e] *= f;
                    }
                m = squares() + eps;
            }
            const float s = __builtin_amdgcn_rsqf(m);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (inside(i)) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        // the row first: s w by itself may be beyond fp32 where the row times s is near 1
                        row.a[i][e] = row.a[i][e] * s * (!APPEND && row.second ? wa[1][i][e] : wa[0][i][e]);
                        row.c[i][e] = row.c[i][e] * s * (!APPEND && row.second ? wc[1][i][e] : wc[0][i][e]);
                    }
                }
        }
        if (APPEND && !row.out)
            return;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (!inside(i))
                continue;
            float v[2 * VEC], o[2 * VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[e] = o[e] = row.a[i][e];
                v[VEC + e] = o[VEC + e] = row.c[i][e];
            }
            if (turned(row.second, i)) {
                const float2 *cs = turn + row.t * half + VEC * (l + LPR * i);
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
            }
            store_unit<VEC>(row.out + unit_a(row.second, i), o);
            store_unit<VEC>(row.out + unit_c(row.second, i), o + VEC);
        }
    };
    constexpr int kGroups = kThreads / LPR;
    int t = group / rows, r = group - t * rows;
    if (t >= here)
        return;
    Row now = fetch(t, r);
    for (;;) {
        for (r += kGroups; r >= rows && t < here; ++t) r -= rows;
        const bool more = t < here;
        Row next;
        if (more)
            next = fetch(t, r);
        finish(now);
        if (!more)
            return;
        now = next;
    }
}

template <int VEC, int LPR, int ITEMS>
hipError_t launch(const RotaryParams &p, hipStream_t stream)
{
    // tokens a workgroup: those that fill its lanes once, and of many tokens up to
    // four times, so that loads of a row run beside the one before
    const int64_t rows = p.first + p.second, fill = kThreads / LPR, tokens = p.B * p.T;
    const int64_t most = std::min(fill, static_cast<int64_t>(kThreads * VEC * ITEMS) / std::max(1, p.positions ? p.R / 2 : 1));
    int64_t per_wg = rows >= fill ? 1 : fill / rows;
    while (tokens / per_wg > kManyBlocks && 2 * per_wg <= most && per_wg * rows < kDepth * fill) per_wg *= 2;
    const int64_t blocks = (tokens + per_wg - 1) / per_wg;
    if (!grid_fits(blocks, kThreads))
        return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (p.slots)
        rotary_kernel<VEC, LPR, ITEMS, true><<<grid, dim3(kThreads), 0, stream>>>(p, static_cast<int>(per_wg));
    else
        rotary_kernel<VEC, LPR, ITEMS, false><<<grid, dim3(kThreads), 0, stream>>>(p, static_cast<int>(per_wg));
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
