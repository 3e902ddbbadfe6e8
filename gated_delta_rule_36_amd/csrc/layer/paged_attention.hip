// Attention of one new token per sequence over a paged cache:
//   out = sum_t p_t v_t,  p = softmax over the visible t of scale q . k_t
// K and V of the visible tokens are read once and bound it; the products run
// beside on matrix instructions for up to 16 query heads of a key head at once.
//
// A wave takes (sequence, key head, 16 of its query heads, split of the tokens)
// and walks tiles of 32 tokens with the running maximum and sum of a softmax,
// nothing shared: no barrier stands in its loop, and with three waves a SIMD at 128 channels
// the next tile's K, V and page numbers are on their way in registers while this one is
// multiplied.  Neighbouring waves take the key heads of the same tokens, which
// lie side by side in the usual cache; with waves of one head next to each
// other the same bytes came at 4.8 TB/s against 5.7 of a cache that keeps a head's
// tokens together.  With few tokens in all, a workgroup's four waves
// share a split and join in LDS instead.  Splits of one sequence leave unnormalised
// results, which a second launch joins.  64 sequences of 8 key heads and 32 query heads,
// 128 channels, 1048576 tokens in all: 804 to 822 us (5.3 TB/s), the rate of a large copy; one of
// 131071 tokens, 2 key heads 35 us (3.8 TB/s; 5.0 in the first of its two launches).
//
// Operands of v_mfma_f32_16x16x32_bf16: lane (r = lane % 16, g = lane / 16)
// holds row / column r, slots 8 g .. 8 g + 7; accumulator register i is row
// 4 g + i of column r.
//   scores^T [token][head] = K Q^T: rows of K and Q are operands as they lie,
//     slot 8 g + e of step s is channel 32 s + 8 g + e;
//   out^T [channel][head] = V^T P^T over the tile's 32 tokens: the scores'
//     accumulators are the operand as they stand, slot 8 g + 4 a + i being token
//     16 a + 4 g + i, and V comes in the same order from LDS by reads that
//     transpose.
// Probabilities enter as three bf16 parts, the first two cut from just below the
// number, so that all are positive and an infinite v stays one (down to 2^-112, where
// the last leaves bf16's numbers).  A part leaves less
// than 1.25 2^-7 of what it is taken from, counted by powers of two, the last one half
// a step, 2^-9, of that: 1.25 2^-23 in all, next to nothing beside fp32's own
// roundings, and out is off by its rounding alone.  The products have time to spare:
// with two parts, good to 2^-16, every time measured here was the same within 1 %.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, TOK = 32;  // tokens of a wave's tile
constexpr int ROWS = static_cast<int>(kAttentionRows);
constexpr float kBelow = 1.0f - 0x1p-10f;
constexpr float kLn2F = 0.693147180559945f;
constexpr float kLowest = -3.402823466e38f, kLargest = 3.402823466e38f;

// The upper halves of two numbers: cut to bf16 towards zero.
__device__ __forceinline__ uint32_t cut_bf16x2(float a, float b)
{
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
}
// e^(x - top).  The difference comes first: scores stay as the scale leaves them, so
// that every one that fp32 holds counts as it is; times log2(e) those above 2.36e38,
// or a scale that large by itself, would be infinite.
//   top itself is a number: taken off from what is infinite it leaves that infinite,
// so scores of -inf weigh nothing and a score of inf makes the sum so.
__device__ __forceinline__ float number(float top) { return __builtin_amdgcn_fmed3f(top, kLowest, kLargest); }
__device__ __forceinline__ float weight(float x, float top) { return exp2_f32((x - top) * kLog2eF); }
// The largest (the sum) over the four lanes of a column.
__device__ __forceinline__ float column_max(float x)
{
    uint32_t u = __float_as_uint(x);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    uint32_t r0 = r[0], r1 = r[1];
    u = __float_as_uint(fmaxf(__uint_as_float(r0), __uint_as_float(r1)));
    r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    r0 = r[0];
    r1 = r[1];
    return fmaxf(__uint_as_float(r0), __uint_as_float(r1));
}
__device__ __forceinline__ float column_sum(float x)
{
    uint32_t u = __float_as_uint(x);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    uint32_t r0 = r[0], r1 = r[1];
    u = __float_as_uint(__uint_as_float(r0) + __uint_as_float(r1));
    r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    r0 = r[0];
    r1 = r[1];
    return __uint_as_float(r0) + __uint_as_float(r1);
}

// The visible tokens [first, first + count) of a sequence; its splits from `used`
// on have none.
struct Visible {
    int first, count, used;
};
__device__ __forceinline__ Visible visible(const AttentionParams &p, int64_t n)
{
    const int64_t room = p.width * static_cast<int64_t>(p.page_size);
    int64_t length = p.lengths[n];
    length = length < 0 ? 0 : length > room ? room : length;
    const int64_t first = p.window > 0 && length > p.window ? length - p.window : 0;
    Visible v;
    v.first = static_cast<int>(first);
    v.count = static_cast<int>(length - first);
    v.used = static_cast<int>((static_cast<uint32_t>(v.count) + static_cast<uint32_t>(p.chunk) - 1) / static_cast<uint32_t>(p.chunk));
    return v;
}

// SHARED: a workgroup's waves share its (sequence, key head, split) and join in
// LDS; otherwise each has its own.  KS steps of 32 channels; a head of D channels
// half fills the last one, or all of it.
// Waves a SIMD by what the registers hold without spilling: of 224 channels two (64
// requests, 65536 tokens in all, 8 key heads 126 us, 149 with one), of 256 one (156; two
// spill 24 registers and take 170, and 170 against 137 for 16, 262144 tokens and 2 key heads).
template <int KS, bool SHARED>
__global__ __launch_bounds__(kThreads, KS <= 4 ? 3 : KS <= 7 ? 2 : 1) void paged_attention_kernel(AttentionParams p, int row_tiles, int64_t items)
{
    constexpr int D = 32 * KS, kPitch = D + 16, kOutPitch = D + 4;
    __shared__ union {
        alignas(16) uint16_t v[kWaves][TOK][kPitch];
        alignas(16) float out[SHARED ? kWaves : 1][ROWS][kOutPitch];
    } sh;
    __shared__ float shared_top[kWaves][ROWS], shared_sum[kWaves][ROWS];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // consecutive items: the key heads of a split, whose rows lie side by side
    if (!SHARED && static_cast<int64_t>(blockIdx.x) * kWaves + wave >= items)
        return;
    uint32_t at = SHARED ? blockIdx.x : blockIdx.x * kWaves + wave;
    const int ht = at % static_cast<uint32_t>(row_tiles);
    at /= static_cast<uint32_t>(row_tiles);
    const int hk = at % static_cast<uint32_t>(p.Hk);
    at /= static_cast<uint32_t>(p.Hk);
    const int split = at % static_cast<uint32_t>(p.splits);
    const int64_t n = at / static_cast<uint32_t>(p.splits);
    constexpr int kStep = SHARED ? kWaves * TOK : TOK;
    const Visible vis = visible(p, n);
    if (split > 0 && split >= vis.used)
        return;
    const int64_t from = static_cast<int64_t>(vis.first) + static_cast<int64_t>(split) * p.chunk;
    const int64_t last = static_cast<int64_t>(vis.first) + vis.count;
    const int t0 = static_cast<int>(from), t1 = static_cast<int>(last < from + p.chunk ? last : from + p.chunk);
    const int group = static_cast<int>(p.Hq / p.Hk), width = static_cast<int>(p.D);
    const int row0 = ht * ROWS, rows = group - row0 < ROWS ? group - row0 : ROWS;

    u32x4_t q[KS];
    const uint16_t *qs = p.q + n * p.qr + (static_cast<int64_t>(hk) * group + row0 + r) * p.D + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        q[s] = u32x4_t{0, 0, 0, 0};
        if (r < rows && 32 * s + 8 * g < width)  // 8 channels of a multiple of 16
            q[s] = *reinterpret_cast<const u32x4_a2 *>(qs + 32 * s);
    }

    const int32_t *table = p.table + n * p.table_stride;
    const uint16_t *kh = p.k + static_cast<int64_t>(hk) * p.ks.head + 8 * g, *vh = p.v + static_cast<int64_t>(hk) * p.vs.head + 8 * g;
    const auto page_index = [&](int t) {
        return p.page_size == 1 ? static_cast<uint32_t>(t) : __umulhi(static_cast<uint32_t>(t), p.page_mul) >> p.page_shift;
    };
    // A lane's tokens of a tile are r and 16 + r; their pages are looked up a tile
    // ahead, as far as the table goes.
    const int room = static_cast<int>(p.width * static_cast<int64_t>(p.page_size));
    int page[2];
    const auto look_up = [&](int base) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int t = base + 16 * a + r;
            page[a] = t < room ? table[page_index(t)] : -1;
        }
    };
    // Of a last step that the head only half fills, the lanes past it read its
    // first channels: what those give K is taken out, rows of V^T there are not stored.
    const bool past = 32 * (KS - 1) + 8 * g >= width;
    const int last_step = past ? -8 * g : 32 * (KS - 1);
    u32x4_t kt[2][KS], vt[2][KS];
    uint32_t seen = 0, ever = 0;  // bit t: token t of the tile (of any tile) is visible
    const auto load_half = [&](int t, int pg, u32x4_t (&kx)[KS], u32x4_t (&vx)[KS]) {
        const u32x4_t none = {0, 0, 0, 0};
        const bool in = t < t1 && pg >= 0 && pg < p.pages;
#pragma unroll
        for (int s = 0; s < KS; ++s) kx[s] = vx[s] = none;
        if (in) {
            const uint32_t off = static_cast<uint32_t>(t) - page_index(t) * p.page_size;
            const uint16_t *kp = kh + static_cast<int64_t>(pg) * p.ks.page + static_cast<int64_t>(off) * p.ks.token;
            const uint16_t *vp = vh + static_cast<int64_t>(pg) * p.vs.page + static_cast<int64_t>(off) * p.vs.token;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                kx[s] = *reinterpret_cast<const u32x4_a2 *>(kp + (s + 1 < KS ? 32 * s : last_step));
                vx[s] = *reinterpret_cast<const u32x4_a2 *>(vp + (s + 1 < KS ? 32 * s : last_step));
            }
        }
        return static_cast<uint32_t>(__ballot(in)) & 0xffffu;
    };
    const auto load = [&](int base) {
        const uint32_t low = load_half(base + r, page[0], kt[0], vt[0]);
        seen = low | load_half(base + 16 + r, page[1], kt[1], vt[1]) << 16;
        ever |= seen;
    };

    f32x4_t o[2 * KS];
#pragma unroll
    for (int d = 0; d < 2 * KS; ++d) o[d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float top = -__builtin_inff(), sum = 0.0f;
    const uint32_t vaddr = lds_addr(&sh.v[wave][4 * g + r / 4][4 * (r & 3)]);

    int base = t0 + (SHARED ? wave * TOK : 0);
    if (base < t1) {
        look_up(base);
        load(base);
        look_up(base + kStep);
    }
    for (; base < t1; base += kStep) {
        f32x4_t score0 = {0.0f, 0.0f, 0.0f, 0.0f}, score1 = score0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (s + 1 == KS && past)
                kt[0][s] = kt[1][s] = u32x4_t{0, 0, 0, 0};
            score0 = mfma(kt[0][s], q[s], score0);
            score1 = mfma(kt[1][s], q[s], score1);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                *reinterpret_cast<u32x4_t *>(&sh.v[wave][16 * a + r][32 * s + 8 * g]) = vt[a][s];
        const uint32_t mine = seen >> (4 * g);
        if (base + kStep < t1) {
            load(base + kStep);
            look_up(base + 2 * kStep);
        }
        float most = -__builtin_inff(), x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float score = (j < 4 ? score0[j & 3] : score1[j & 3]) * p.scale;
            x[j] = mine >> (j < 4 ? j : 12 + j) & 1 ? score : -__builtin_inff();
            most = fmaxf(most, x[j]);
        }
        const float next = fmaxf(top, column_max(most));
        const float from_top = number(next);
        const float keep = weight(number(top), from_top);
        top = next;
        sum *= keep;
        u32x4_t hi, mid, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = weight(x[2 * j], from_top), b = weight(x[2 * j + 1], from_top);
            sum += a + b;
            const uint32_t h = cut_bf16x2(a * kBelow, b * kBelow);
            hi[j] = h;
            const float rest_a = a - lo_f32(h), rest_b = b - hi_f32(h);  // exact, as what is left of them
            const uint32_t m = cut_bf16x2(rest_a * kBelow, rest_b * kBelow);
            mid[j] = m;
            lo[j] = pack_bf16x2(rest_a - lo_f32(m), rest_b - hi_f32(m));
        }
        if (__any(keep != 1.0f)) {
#pragma unroll
            for (int d = 0; d < 2 * KS; ++d) o[d] *= keep;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int d = 0; d < 2 * KS; ++d) {
            const u32x2_t x = lds_tr(vaddr + 32 * d), y = lds_tr(vaddr + 32 * d + 32 * kPitch);
            const u32x4_t va = {x[0], x[1], y[0], y[1]};
            o[d] = mfma(va, hi, o[d]);
            o[d] = mfma(va, mid, o[d]);
            o[d] = mfma(va, lo, o[d]);
        }
        asm volatile("" ::: "memory");
    }

    sum = column_sum(sum);
    // Scores that are all -inf leave no weight to divide by, NaN; only a row without a visible token is 0.  The lowest
    // number tells them apart from here on, and beside any score in other splits it comes to nothing.
    if (ever != 0 && top == -__builtin_inff())
        top = kLowest;
    if constexpr (SHARED) {
        // the waves' results, one after the other in LDS; each goes on with a quarter of the channels
        __syncthreads();
        if (g == 0) {
            shared_top[wave][r] = top;
            shared_sum[wave][r] = sum;
        }
#pragma unroll
        for (int d = 0; d < 2 * KS; ++d) *reinterpret_cast<f32x4_t *>(&sh.out[wave][r][16 * d + 4 * g]) = o[d];
        __syncthreads();
        float most = shared_top[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) most = fmaxf(most, shared_top[w][r]);
        const float from_top = number(most);
        float f[kWaves];
        top = most;
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            f[w] = weight(shared_top[w][r], from_top);
            sum = fmaf(f[w], shared_sum[w][r], sum);
        }
#pragma unroll
        for (int d = 0; d < 2 * KS; ++d)
            if ((d & (kWaves - 1)) == wave) {
                o[d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) o[d] += f[w] * *reinterpret_cast<const f32x4_t *>(&sh.out[w][r][16 * d + 4 * g]);
            }
    }
    const auto mine = [&](int d) { return 16 * d < width && (!SHARED || (d & (kWaves - 1)) == wave); };
    const bool first = g == 0 && (!SHARED || wave == 0);
    if (r >= rows)
        return;
    const int64_t head = n * p.Hq + static_cast<int64_t>(hk) * group + row0 + r;
    if (vis.used <= 1) {
        const bool none = top == -__builtin_inff();
        const float f = none ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int d = 0; d < 2 * KS; ++d)
            if (mine(d))
                *reinterpret_cast<u32x2_t *>(p.out + head * p.D + 16 * d + 4 * g) =
                    u32x2_t{pack_bf16x2(o[d][0] * f, o[d][1] * f), pack_bf16x2(o[d][2] * f, o[d][3] * f)};
        if (first && p.lse)
            p.lse[head] = none ? top : fmaf(log2f(sum), kLn2F, top);
    } else {
        const int64_t slot = head * p.splits + split;
#pragma unroll
        for (int d = 0; d < 2 * KS; ++d)
            if (mine(d))
                *reinterpret_cast<f32x4_t *>(p.part + slot * p.D + 16 * d + 4 * g) = o[d];
        if (first) {
            p.stats[2 * slot] = top;
            p.stats[2 * slot + 1] = sum;
        }
    }
}

// Joins the splits of a row: LANES lanes of four channels each, the splits dealt
// over the workgroup's groups of lanes, each of which keeps a running maximum
// and sum of its own; they meet in LDS.  A workgroup takes 4 LANES channels: 32 of
// a row of many splits, so that several share it, all of one of few (64
// requests of up to 65 splits, 32 heads: 15 us by 32 channels, 7 by 128; one of
// 1024 splits and 16 heads 8 by 32 channels).
constexpr int kJoinThreads = 256;
template <int LANES>
__global__ __launch_bounds__(kJoinThreads) void paged_attention_join_kernel(AttentionParams p, int parts)
{
    constexpr int GROUPS = kJoinThreads / LANES;
    __shared__ __align__(16) float part[GROUPS][4 * LANES];
    __shared__ float tops[GROUPS], sums[GROUPS];
    const uint32_t head = blockIdx.x / static_cast<uint32_t>(parts), at = blockIdx.x - head * static_cast<uint32_t>(parts);
    const Visible vis = visible(p, head / static_cast<uint32_t>(p.Hq));
    if (vis.used <= 1)
        return;
    const int tid = threadIdx.x, grp = tid / LANES, l = tid % LANES, d = 4 * LANES * static_cast<int>(at) + 4 * l;
    const bool here = d < p.D;
    const float *stats = p.stats + 2 * head * p.splits, *src = p.part + head * p.splits * p.D + (here ? d : 0);
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    float top = -__builtin_inff(), total = 0.0f;
#pragma unroll 4
    for (int s = grp; s < vis.used; s += GROUPS) {
        const float m = stats[2 * s], next = fmaxf(top, m), from_top = number(next);
        const float keep = weight(number(top), from_top), f = weight(m, from_top);
        total = fmaf(f, stats[2 * s + 1], total * keep);
        x = f * *reinterpret_cast<const f32x4_t *>(src + s * p.D) + x * keep;
        top = next;
    }
    *reinterpret_cast<f32x4_t *>(&part[grp][4 * l]) = x;
    if (l == 0) {
        tops[grp] = top;
        sums[grp] = total;
    }
    __syncthreads();
    if (tid >= LANES || !here)
        return;
    float most = tops[0];
    for (int k = 1; k < GROUPS; ++k) most = fmaxf(most, tops[k]);
    const float from_top = number(most);
    x = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    total = 0.0f;
#pragma unroll 4
    for (int k = 0; k < GROUPS; ++k) {
        const float f = weight(tops[k], from_top);
        total = fmaf(f, sums[k], total);
        x += f * *reinterpret_cast<const f32x4_t *>(&part[k][4 * l]);
    }
    const bool none = most == -__builtin_inff();
    const float f = none ? 0.0f : 1.0f / total;
    *reinterpret_cast<u32x2_t *>(p.out + head * p.D + d) =
        u32x2_t{pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f)};
    if (d == 0 && p.lse)
        p.lse[head] = none ? most : fmaf(log2f(total), kLn2F, most);
}

template <int LANES>
hipError_t launch_join(const AttentionParams &p, hipStream_t stream)
{
    const int64_t parts = (p.D + 4 * LANES - 1) / (4 * LANES);
    paged_attention_join_kernel<LANES><<<dim3(static_cast<uint32_t>(p.N * p.Hq * parts)), dim3(kJoinThreads), 0, stream>>>(
        p, static_cast<int>(parts));
    return hipGetLastError();
}

template <int KS>
hipError_t launch(const AttentionParams &p, hipStream_t stream)
{
    const int64_t row_tiles = (p.Hq / p.Hk + ROWS - 1) / ROWS;
    const int64_t items = p.N * p.splits * row_tiles * p.Hk, blocks = p.shared ? items : (items + kWaves - 1) / kWaves;
    if (!grid_fits(blocks, kThreads))  // of several splits N Hq is at most 2^18: the join fits then
        return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (p.shared)
        paged_attention_kernel<KS, true><<<grid, dim3(kThreads), 0, stream>>>(p, static_cast<int>(row_tiles), items);
    else
        paged_attention_kernel<KS, false><<<grid, dim3(kThreads), 0, stream>>>(p, static_cast<int>(row_tiles), items);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    return p.splits > 128 ? launch_join<8>(p, stream) : p.D <= 128 ? launch_join<32>(p, stream) : launch_join<64>(p, stream);
}

}  // namespace

hipError_t launch_paged_attention(const AttentionParams &p, hipStream_t stream)
{
    switch ((p.D + 31) / 32) {
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
