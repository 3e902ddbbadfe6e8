// Short causal depthwise convolution with its activation and, for query and
// key heads, their L2 norm:
//   y[t,c] = act(bias[c] + sum_j w[c,j] x[t - W + 1 + j, c]),  j = 0 .. W-1
//   out    = y, or y / sqrt(sum over its group of y^2 + eps)
// Inputs before a sequence's first token come from its state, the last W - 1
// inputs of what came before (oldest first).
//
// Every input is needed W times and the arithmetic is about 2 W operations a
// cell against 4 bytes, so memory bounds it.  One wave owns 512 channels
// (eight a lane, 16-byte loads) of one tile of consecutive tokens and slides
// the window through registers: a row is read once per tile, plus W - 1 rows
// in front of the tile.  No LDS, no barriers; waves are independent.
//
// The tile at a sequence's start reads the initial state and also writes the
// final one (each channel by the lane that owns it, after its read), so the two
// may be one buffer.
//
// Tiles are 16 tokens long (one row in six read twice, from the caches), or 8
// where longer ones would leave fewer than kFew waves: packed prompts of 19595
// tokens and 4096 channels take 70.5 us with 16, 72.6 with 8 and 80 with 32; 4097
// tokens of 1283 channels 9.0 us with 8, 11.3 with 16 and 18.3 with 32.
//
// One token of 64 rows of 12288 channels takes 8.1 us where memory would take 2.5:
// state, input and weights are asked for one after the other, and four rows are
// computed for the one.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kWaves = 4;
constexpr int kBatch = 4;  // rows in flight
constexpr int64_t kFew = 4096;  // waves, at 32 tokens a tile

template <int W>
__global__ __launch_bounds__(64 * kWaves) void conv_kernel(ConvParams p, uint32_t tasks, uint32_t cblocks, uint32_t tile_len)
{
    const int lane = threadIdx.x & 63;
    const uint32_t task = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
    if (task >= tasks)
        return;
    const uint32_t slot = task / cblocks, cb = task - slot * cblocks;
    const Tile tile = find_tile(p.seqs, tile_len, slot);
    const int64_t c0 = (static_cast<int64_t>(cb) * 64 + lane) * 8;
    if (!tile.valid || c0 >= p.D)
        return;
    const Eight ch = eight_of(c0, p.D);

    const int64_t len = tile.end - tile.begin;
    const int64_t t0 = static_cast<int64_t>(tile.index) * tile_len, t1 = t0 + tile_len < len ? t0 + tile_len : len;
    const uint16_t *x = p.x + tile.row * p.xb + static_cast<int64_t>(tile.begin) * p.xt;  // token 0 of the sequence
    uint16_t *out = p.out + (tile.row * p.seqs.T + tile.begin) * p.D;

    float win[W - 1 + kBatch][8];  // rows t - W + 1 .. t + kBatch - 1
    if (tile.index == 0) {
#pragma unroll
        for (int m = 0; m < W - 1; ++m) {
            if (p.init_state) {
                load8(p.init_state, p.init_kind, (tile.n * (W - 1) + m) * p.D, ch, win[m]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) win[m][e] = 0.0f;
            }
        }
        if (p.final_state) {
            // row m of the final state is input len - (W - 1) + m
#pragma unroll
            for (int m = 0; m < W - 1; ++m) {
                float f[8];
                if (len + m >= W - 1) {
                    unpack8(load8_raw(x + (len + m - (W - 1)) * p.xt, ch), f);
                } else {
#pragma unroll
                    for (int q = 0; q < W - 1; ++q)
                        if (len + m == q) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] = win[q][e];
                        }
                }
                store8(p.final_state, p.final_kind, (tile.n * (W - 1) + m) * p.D, ch, f);
            }
        }
    } else {
#pragma unroll
        for (int m = 0; m < W - 1; ++m) unpack8(load8_raw(x + (t0 - (W - 1) + m) * p.xt, ch), win[m]);
    }
    if (t0 >= t1)
        return;

    float w[W][8], bias[8];
    {
        // the lane's W x 8 weights lie together: element e of channel c at 8 W consecutive places
        float flat[W * 8];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int left = ch.count * W - 8 * j;  // of a row of fewer than eight channels
            const Eight piece = {ch.at * W + 8 * j, 0, ch.count == 8 || left > 8 ? 8 : (left > 0 ? left : 0)};
            load8(p.weight, p.weight_kind, 0, piece, flat + 8 * j);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) w[j][e] = flat[e * W + j];
    }
    if (p.bias) {
        load8(p.bias, p.weight_kind, 0, ch, bias);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = 0.0f;
    }

    for (int64_t t = t0; t < t1; t += kBatch) {
        u32x4_t raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) raw[i] = load8_raw(x + (t + i < t1 ? t + i : t1 - 1) * p.xt, ch);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            unpack8(raw[i], win[W - 1 + i]);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) y[e] = fmaf(w[j][e], win[i + j][e], y[e]);
            }
            if (p.act == kActSilu) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = silu_f32(y[e]);
            }
            if (p.l2norm) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
                const auto group_sum = [&](float v) {
                    return p.l2norm == 64 ? lane_sum<8>(v) : p.l2norm == 128 ? lane_sum<16>(v) : lane_sum<32>(v);
                };
                ss = group_sum(ss);
                float m = ss + p.l2eps.plain;
                if (__any(!norm_in_range(m))) {  // the wave together: the sum below is over lanes
                    const float f = norm_in_range(m) ? 1.0f : norm_shift(m), eps = norm_in_range(m) ? p.l2eps.plain : shifted_eps(p.l2eps, m);
                    ss = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y[e] *= f;
                        ss = fmaf(y[e], y[e], ss);
                    }
                    m = group_sum(ss) + eps;
                }
                const float r = __builtin_amdgcn_rsqf(m);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= r;
            }
            if (t + i < t1)
                store8_raw(out + (t + i) * p.D, pack8(y), ch);
        }
#pragma unroll
        for (int m = 0; m < W - 1; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) win[m][e] = win[m + kBatch][e];
    }
}

template <int W>
hipError_t launch(const ConvParams &p, hipStream_t stream)
{
    const int64_t cblocks = (p.D + 511) / 512;
    const int64_t len = tile_slots(p.seqs, 32) * cblocks < kFew ? 8 : 16, tasks = tile_slots(p.seqs, len) * cblocks;
    const int64_t blocks = (tasks + kWaves - 1) / kWaves;
    if (!grid_fits(blocks, 64 * kWaves))
        return hipErrorInvalidConfiguration;
    conv_kernel<W><<<dim3(static_cast<uint32_t>(blocks)), dim3(64 * kWaves), 0, stream>>>(
        p, static_cast<uint32_t>(tasks), static_cast<uint32_t>(cblocks), static_cast<uint32_t>(len));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv(const ConvParams &p, int W, hipStream_t stream)
{
    switch (W) {
    case 1: return launch<1>(p, stream);
    case 2: return launch<2>(p, stream);
    case 3: return launch<3>(p, stream);
    case 4: return launch<4>(p, stream);
    case 5: return launch<5>(p, stream);
    case 6: return launch<6>(p, stream);
    case 7: return launch<7>(p, stream);
    case 8: return launch<8>(p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace layer
}  // namespace kda
