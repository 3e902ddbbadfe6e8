// Device helpers shared by the layer kernels: eight-element loads and stores
// at any element alignment, sums over lanes, and the map from work slots to
// sequences.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_device.h"
#include "layer_internal.h"

namespace kda {
namespace layer {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
// The same sixteen bytes at element alignment: rows of odd widths and slices
// of fused projections start anywhere.  Global memory serves unaligned
// 16-byte accesses directly, so one code path covers every stride.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b)
{
    const bf16x2_t v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ void unpack8(u32x4_t u, float f[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = lo_f32(u[i]);
        f[2 * i + 1] = hi_f32(u[i]);
    }
}
__device__ __forceinline__ u32x4_t pack8(const float f[8])
{
    return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7])};
}

// The eight elements a lane takes of a row of `size`: from `at` on.  The last
// lane of a row whose size is no multiple of eight steps back to the row's
// last eight and does not own the first `skip` of them (eight, for a lane past
// the row): loads are whole wherever the row holds eight elements, so no lane
// waits for its own single ones, and only stores go one by one.  A row of
// fewer than eight has one lane that owns `size` elements, loaded singly.
struct Eight {
    int64_t at;
    int skip, count;  // elements skip .. count - 1 are the lane's
};
__device__ __forceinline__ Eight eight_of(int64_t at, int64_t size)
{
    Eight v = {at, 0, 8};
    if (size < 8) {
        v.at = 0;
        v.count = static_cast<int>(size);
        v.skip = at == 0 ? 0 : v.count;
    } else if (at + 8 > size) {
        v.at = size - 8;
        v.skip = at < size ? static_cast<int>(at + 8 - size) : 8;
    }
    return v;
}
__device__ __forceinline__ bool owns(const Eight &v, int e) { return e >= v.skip && e < v.count; }

// Zero for what is not the lane's, whatever lies there.
__device__ __forceinline__ void keep_own(const Eight &v, float f[8])
{
    if (v.skip == 0 && v.count == 8)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (!owns(v, i))
            f[i] = 0.0f;
}

__device__ __forceinline__ u32x4_t load8_raw(const uint16_t *p, const Eight &v)
{
    if (v.count == 8)
        return *reinterpret_cast<const u32x4_a2 *>(p + v.at);
    u32x4_t u = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < v.count)
            u[i / 2] |= static_cast<uint32_t>(p[v.at + i]) << (16 * (i & 1));
    return u;
}
__device__ __forceinline__ void store8_raw(uint16_t *p, u32x4_t u, const Eight &v)
{
    if (v.skip == 0 && v.count == 8) {
        *reinterpret_cast<u32x4_a2 *>(p + v.at) = u;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (owns(v, i))
            p[v.at + i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
}
// The same of kind `kind`, as fp32; `base` at element `row`.
__device__ __forceinline__ void load8(const void *base, int kind, int64_t row, const Eight &v, float f[8])
{
    if (kind == kBf16) {
        unpack8(load8_raw(static_cast<const uint16_t *>(base) + row, v), f);
        return;
    }
    const float *p = static_cast<const float *>(base) + row + v.at;
    if (v.count == 8) {
        const f32x4_t a = *reinterpret_cast<const f32x4_a4 *>(p), b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < v.count ? p[i] : 0.0f;
}
__device__ __forceinline__ void store8(void *base, int kind, int64_t row, const Eight &v, const float f[8])
{
    if (kind == kBf16) {
        store8_raw(static_cast<uint16_t *>(base) + row, pack8(f), v);
        return;
    }
    float *p = static_cast<float *>(base) + row + v.at;
    if (v.skip == 0 && v.count == 8) {
        *reinterpret_cast<f32x4_a4 *>(p) = f32x4_t{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f32x4_a4 *>(p + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (owns(v, i))
            p[i] = f[i];
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
// The sum over aligned groups of L lanes (1..64, a power of two), in every
// lane: quad permutations, the half-row and row mirrors, then exchanges of
// 16-lane rows and of wave halves.  All lanes of the group must be active.
template <int L>
__device__ __forceinline__ float lane_sum(float x)
{
    if constexpr (L >= 2) x = dpp_add<0xb1>(x);
    if constexpr (L >= 4) x = dpp_add<0x4e>(x);
    if constexpr (L >= 8) x = dpp_add<0x141>(x);
    if constexpr (L >= 16) x = dpp_add<0x140>(x);
    if constexpr (L >= 32) {
        const uint32_t u = __float_as_uint(x);
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const uint32_t r0 = r[0], r1 = r[1];
        x = __uint_as_float(r0) + __uint_as_float(r1);
    }
    if constexpr (L >= 64) {
        const uint32_t u = __float_as_uint(x);
        const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        const uint32_t r0 = r[0], r1 = r[1];
        x = __uint_as_float(r0) + __uint_as_float(r1);
    }
    return x;
}

__device__ __forceinline__ float silu_f32(float x) { return x * sigmoid_f32(x); }

// Norms divide by the root of m, a sum or mean of squares and eps.  Where fp32
// does not hold the squares (m infinite, or so small that some may be denormal,
// which the reciprocal root takes for 0) the numbers are scaled by a power of two
// and squared again: by 2^94 below m = 2^-80, so that 16384 squares stay under
// 2^122 and that of the least number above 2^-124, else by 2^-80.
__device__ __forceinline__ bool norm_in_range(float m) { return m >= 0x1p-80f && m < __builtin_inff(); }
__device__ __forceinline__ float norm_shift(float m) { return m < 0x1p-80f ? 0x1p94f : 0x1p-80f; }
__device__ __forceinline__ float shifted_eps(const NormEps &e, float m) { return m < 0x1p-80f ? e.up : e.down; }

// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v|, or v itself above `plain`:
// 20, where the two agree in fp32, or below everything for steps that are not
// to be transformed.  Most steps are far below 1, so u and its log1p have to be
// good relative to themselves: the product |v| log2(e) is carried to twice its
// digits, and log1p(u) = 2 artanh(u / (2 + u)) as its series in z = u / (2 + u)
// <= 1/3 (z^15 / 15 left out, 1e-8 of the sum).  A few 2^-24 in all.
__device__ __forceinline__ float dt_plain_above(int softplus) { return softplus ? 20.0f : -__builtin_inff(); }
__device__ __forceinline__ float softplus_f32(float v, float plain)
{
    const float n = v < -150.0f ? -150.0f : -fabsf(v), hi = n * kLog2eF;  // e^-150 is 0
    const float lo = fmaf(n, 1.92596303e-8f, fmaf(n, kLog2eF, -hi));  // log2(e) = kLog2eF + 1.93e-8
    const float e = exp2_f32(hi), u = fmaf(e, lo * 0.693147181f, e);
    const float z = u * __builtin_amdgcn_rcpf(2.0f + u), w = z * z;
    float s = fmaf(w, 1.0f / 13, 1.0f / 11);
    s = fmaf(w, s, 1.0f / 9);
    s = fmaf(w, s, 1.0f / 7);
    s = fmaf(w, s, 1.0f / 5);
    s = fmaf(w, s, 1.0f / 3);
    s = 2.0f * fmaf(w * z, s, z);
    return v > plain ? v : fmaxf(v, 0.0f) + s;
}

// The sum over the wave's lanes up to and with each lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_plus(uint32_t x)
{
    return x + static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ uint32_t prefix64(uint32_t x)
{
    x = dpp_plus<0x118, 0xf>(dpp_plus<0x114, 0xf>(dpp_plus<0x112, 0xf>(dpp_plus<0x111, 0xf>(x))));
    return dpp_plus<0x143, 0xc>(dpp_plus<0x142, 0xa>(x));  // lane 15 of rows 0, 2 to 1, 3; lane 31 to rows 2, 3
}

// Sequences are cut into tiles of `len` tokens that start at the sequence's
// first token, at least one a sequence.  In a batch each has ceil(T / len).
// Of packed ones T / len + N slots hold all tiles, since ceil((b - a) / len)
// <= floor(b / len) - floor(a / len) + 1, so the host can size the grid
// without reading cu_seqlens.  Up to 64 sequences, one a lane, take their
// slots one after the other: the slots that no tile uses are the last ones,
// and the tiles spread evenly over the chip (unused slots between them cost
// the scan of 19595 tokens in 8 sequences up to 40 %: some compute units got
// two of 32 segments).  Of more, sequence n owns the slots from cu[n] / len + n
// on, and a slot finds its sequence by search.
constexpr int64_t kLaneSequences = 64;
struct Tile {
    int64_t n, row;       // sequence, its batch row
    uint32_t begin, end;  // its tokens
    uint32_t index;       // tile within the sequence; its tokens may be none
    bool valid;           // false: a slot no tile uses
};

// Offsets are at most T < 2^31, and so are slots (the grid's limit): all of
// this is 32-bit arithmetic.
__device__ __forceinline__ uint32_t clamp_offset(const Seqs &s, int64_t n)
{
    const int64_t v = s.cu[n];
    return static_cast<uint32_t>(v < 0 ? 0 : (v > s.T ? s.T : v));
}

// Sequence `lane` of at most 64 packed ones: its tokens, its first slot and the
// next one's (lanes past the last sequence: none, after all others).
struct LaneSequence {
    uint32_t begin, end, first, next;
};
__device__ __forceinline__ LaneSequence lane_sequence(const Seqs &s, uint32_t len, uint32_t lane)
{
    LaneSequence q = {0, 0, 0, 0};
    uint32_t count = 0;
    if (lane < s.N) {
        q.begin = clamp_offset(s, lane);
        const uint32_t end = clamp_offset(s, lane + 1);
        q.end = end > q.begin ? end : q.begin;
        count = q.end > q.begin ? (q.end - q.begin + len - 1) / len : 1;
    }
    q.next = prefix64(count);
    q.first = q.next - count;
    return q;
}

__device__ __forceinline__ Tile find_tile(const Seqs &s, uint32_t len, uint32_t slot)
{
    Tile t;
    if (!s.cu) {
        const uint32_t T = static_cast<uint32_t>(s.T), per = T > 0 ? (T + len - 1) / len : 1, n = slot / per;
        t.n = n;
        t.row = n;
        t.index = slot - n * per;
        t.begin = 0;
        t.end = T;
        t.valid = true;
        return t;
    }
    const uint32_t lane = __lane_id();
    t.row = 0;
    if (s.N <= kLaneSequences) {
        const LaneSequence q = lane_sequence(s, len, lane);
        const uint64_t past = __ballot(q.next > slot);
        const int n = past ? __builtin_ctzll(past) : 0;
        t.n = n;
        t.begin = __builtin_amdgcn_readlane(q.begin, n);
        t.end = __builtin_amdgcn_readlane(q.end, n);
        t.index = slot - __builtin_amdgcn_readlane(q.first, n);
        t.valid = past != 0;
        return t;
    }
    // the last n with cu[n] / len + n <= slot; 64 probes a round.  Offsets
    // out of order still end at some n in [0, N).
    uint32_t lo = 0, hi = static_cast<uint32_t>(s.N);
    while (hi - lo > 1) {
        const uint32_t step = (hi - lo + 63) / 64, n = lo + lane * step;
        const bool below = n < hi && clamp_offset(s, n) / len + n <= slot;
        const uint32_t count = __popcll(__ballot(below));
        if (count == 0)
            break;
        lo += (count - 1) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    t.n = lo;
    t.begin = clamp_offset(s, lo);
    t.end = clamp_offset(s, lo + 1);
    if (t.end < t.begin)
        t.end = t.begin;
    const uint32_t first = t.begin / len + lo;
    t.index = slot - first;
    t.valid = slot == first || (slot > first && t.index < (t.end - t.begin + len - 1) / len);
    return t;
}

}  // namespace layer
}  // namespace kda
