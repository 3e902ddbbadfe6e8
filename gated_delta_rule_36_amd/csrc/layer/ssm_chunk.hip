// The selective state space scan in tiles of 64 tokens, two blocks of 32, on
// matrix instructions.  Per head, with a_t = -e^A_log log2(e) dt_t, G_t the
// sum of a over the block up to and with token t, R_t the sum over its tokens
// after t, T the whole block's sum, w_t = dt_t 2^(R_t), and S the state [P, N]
// in front of the tile:
//   first block   y_t = 2^(G_t) S c_t + sum_(s <= t) (c_t . b_s) 2^(G_t - G_s) dt_s x_s
//   second block  y_t = 2^(G_t) (2^(T_0) S c_t + sum_(first block) (c_t . b_s) w_s x_s)
//                       + the same sum over its own tokens
//   out_t = (y_t + D x_t) silu(z_t)
//   S <- 2^(T_1) (2^(T_0) S + sum_0 w_s x_s b_s^T) + sum_1 w_s x_s b_s^T
// Since 2^(G_t - G_s) dt_s = 2^(G_t - T) w_s, the sum over a block's own tokens
// takes the same weighted x as the state: 2^(G_t - T) sum (c_t . b_s) w_s x_s,
// and c b^T, which the heads of a group share, is the other factor.  A gentle
// tile, one that decays by less than 2^-40 in all (and, where steps may be
// negative, neither decays nor grows by more from any token to its end), scales
// its first block's weights and the state to the tile's end at once, so that
// 2^(G_t - T) stays well inside fp32's range.  A steep one goes block by block
// and forms M[t,s] = (c_t . b_s) 2^(G_t - G_s) dt_s itself; no other exponent is
// positive there after softplus, so nothing overflows however strong the decay.
//
// A difference of G loses what a strong decay in the same block rounds away,
// so G is held in fixed point: 32-bit integers in a unit of 2^-29 .. 2^-30 of
// the block's sum of |a|, whose sums and differences are exact.  Decays below
// 2^-160 count as that (both are 0 in fp32), so a unit is at most 2^-17.  R is
// summed in fp32 from the block's end, so that the weights of the newest
// tokens, which make up most of the state, are the most exact.
//
// One wave owns a unit: 32 of a head's P columns, with the fp32 state [32, N]
// in accumulators for a whole segment of the sequence.  A workgroup of eight
// waves takes eight consecutive units of one group (P = 64: four heads), which
// share b, c and c b^T (formed once a tile, 16 x 16 tiles spread over the
// waves).  b, c and x go through registers into LDS, the next tile's loads in
// flight while this one is computed.  x is read from memory once per pass.
//
// What bounds it is vector instructions, and what two waves a SIMD leave
// uncovered (the state takes 64 registers, a tile in flight 32).  A wave's tile
// (P = 64, N = 128) takes 102 matrix instructions and 1519 vector ones, most of
// them to round S, the weighted x and c b^T into their parts; they fill 26 and 53 %
// of a SIMD's cycles.  8 x 16384 tokens of 32 heads, 1.7 GB to move: 900 to 960 us,
// of which the own states take 204 to 225 and joining them 12.  19595 tokens in 8
// sequences 176 to 198 us; one of 8192 tokens with 16 heads of 128 x 64 60 us.
// Asking for the next tile before c b^T is formed gained 5 % over asking after
// it, the priorities below 4 %.  Measured and not better: waves of 16 columns (16
// of them), waves of 64, two workgroups of four waves a compute unit, loads spread
// over the tile, z and out through LDS or exchanged between lanes into whole
// 64-byte rows, more and shorter segments for the own states (13 % slower in twice
// as many), the workgroups of a segment on one L2, stores held back until the next
// tile has arrived (3 to 5 % slower), non-temporal z (10 % slower) and out (3 %).
//
// Operands.  v_mfma_f32_32x32x16_bf16 contracts 16 slots; lane (l32, half)
// holds slots 8 half .. 8 half + 7 of row / column l32, and accumulator
// register r = 4 i + q is row 8 i + 4 half + q.  Which contraction index a
// slot stands for is free as long as both operands agree:
//   over n:  slot e of step (tile, j) is n = 32 tile + 16 j + 8 (e / 4) + 4 half + e % 4,
//            so a state accumulator is the operand as it stands;
//   over s:  slot e of step j is s = 8 (e % 4) + 4 half + 2 j + e / 4, the order
//            of an accumulator over s, and the four tokens a transposing LDS
//            read takes are 8 rows apart, which with rows of 2 mod 16 dwords
//            puts them in distinct banks.
// Row / column l32 of the unit stands for column p = 16 ((l32 >> 2) & 1) +
// 4 (l32 >> 3) + l32 % 4, so that a lane ends with 16 adjacent columns of its
// token's output.
//
// x, b and c are bf16 and enter as they are.  Of the fp32 factors, S, c b^T and
// M enter as two bf16 parts (the value rounded, and the rest rounded: good to
// 2^-17 of itself; out is rounded to 2^-8); the weighted x enters the state as
// three, which hold it whole, at any decay: what a decay leaves of a block is
// all there is of the state where later tokens bring nothing.  (Two for blocks
// that decay by more than 2^-4 were 4 to 8 % faster and left 2^-17.)  Of the
// parts' products with c b^T the last times the last, 2^-18 of the whole, is
// left out.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int CH = static_cast<int>(kSsmChunk);  // tokens a block
constexpr int TM = 2 * CH;                       // tokens a tile
constexpr int NW = static_cast<int>(kSsmWaves);  // waves, units a workgroup
// Log decay from which on a tile is steep.  The gentle way is 12 % faster on
// 4 x 8192 tokens that hardly decay (250 against 283 us); from -80 on it is as fast,
// with less room for small values of S.
constexpr float kSteep = -40.0f;
// Log decay from a block to the segment's end below which nothing earlier is
// left in fp32: what is finite there is 0 times 2^-300, also where negative
// steps (without softplus) let it grow before.
constexpr float kNothing = -300.0f;
// Weights from 2^32 on and x from 2^64 on are looked at one by one (see scrub):
// below, their product is finite.
constexpr float kLargeWeight = 0x1p32f;
template <int V>
struct Int {
    constexpr int operator()() const { return V; }
};
constexpr int kThreads = 64 * NW;
constexpr int kXPitch = NW * 32 + 4;  // bf16 elements of an x row in LDS

__device__ __forceinline__ bf16x8_t cat8(u32x2_t a, u32x2_t b)
{
    return __builtin_bit_cast(bf16x8_t, u32x4_t{a[0], a[1], b[0], b[1]});
}
__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// Nothing is scheduled across this.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }
// x, computed here and not before: what is derived from it inside a loop stays
// there instead of occupying a register through all of it.
__device__ __forceinline__ int here(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}
__device__ __forceinline__ const char *bytes(const uint16_t *p) { return reinterpret_cast<const char *>(p); }
// a b + c over the two bf16 numbers of a and b.
__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t b, float c)
{
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a), __builtin_bit_cast(bf16x2_t, b), c, false);
}
// v as a sum of bf16 numbers, each what is left rounded to nearest: two leave
// 2^-17 of v at most (half a step of 2^-8 v, which is half a step of v), three
// hold its 24 bits.
template <int PARTS>
__device__ __forceinline__ void split8(const float v[8], bf16x8_t parts[PARTS])
{
    static_assert(PARTS == 2 || PARTS == 3, "two parts or three");
    u32x4_t h[PARTS];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            h[k][i] = pack_bf16x2(a, b);
            a -= lo_f32(h[k][i]);
            b -= hi_f32(h[k][i]);
        }
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k) parts[k] = __builtin_bit_cast(bf16x8_t, h[k]);
}
// The third part of v, which two leave out.
__device__ __forceinline__ bf16x8_t rest8(const float v[8])
{
    u32x4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t first = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        const float a = v[2 * i] - lo_f32(first), b = v[2 * i + 1] - hi_f32(first);
        const uint32_t second = pack_bf16x2(a, b);
        h[i] = pack_bf16x2(a - lo_f32(second), b - hi_f32(second));
    }
    return __builtin_bit_cast(bf16x8_t, h);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_zero(int x)
{
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, true);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_zero(float x)
{
    return __builtin_bit_cast(float, dpp_zero<CTRL, ROWS>(__builtin_bit_cast(int, x)));
}
__device__ __forceinline__ float read_lane(float x, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
// x, the same in all lanes, as worked out up to here.
__device__ __forceinline__ float of_wave(float x)
{
    asm volatile("" : "+v"(x));
    return read_lane(x, 0);
}
// Sums over the 32 lanes of each wave half up to and with each lane.
template <typename V>
__device__ __forceinline__ V prefix32(V x)
{
    x += dpp_zero<0x111, 0xf>(x);
    x += dpp_zero<0x112, 0xf>(x);
    x += dpp_zero<0x114, 0xf>(x);
    x += dpp_zero<0x118, 0xf>(x);
    return x + dpp_zero<0x142, 0xa>(x);  // lane 15 of rows 0, 2 to rows 1, 3
}
// Sums over the lanes of each wave half after each lane.
__device__ __forceinline__ float after32(float x, int lane)
{
    x = dpp_zero<0x130, 0xf>(x);  // the next lane's
    x = (lane & 31) == 31 ? 0.0f : x;
    x += dpp_zero<0x101, 0xf>(x);
    x += dpp_zero<0x102, 0xf>(x);
    x += dpp_zero<0x104, 0xf>(x);
    x += dpp_zero<0x108, 0xf>(x);
    const float r1 = read_lane(x, 16), r3 = read_lane(x, 48);
    return x + ((lane & 16) ? 0.0f : (lane < 32 ? r1 : r3));
}

template <int N, bool OUT>
struct Shared {
    static constexpr int kPitch = N + 4;
    alignas(16) uint16_t b[TM][kPitch];
    alignas(16) uint16_t c[OUT ? TM : 1][kPitch];
    alignas(16) uint16_t x[TM][kXPitch];
    // c_t . b_s as an operand, [rounded, rest][j][half][t][slot]: the first
    // block with itself, the second with itself, the second's t with the first's s
    alignas(16) uint16_t cb[OUT ? 3 : 1][2][2][2][CH][8];
    // per head of the workgroup, for the tiles in turn: G of a token in its
    // block's unit, dt, w; the blocks' T and units
    alignas(16) int g[2][NW][OUT ? TM : 4];
    alignas(16) float d[2][NW][OUT ? TM : 4];
    alignas(16) float w[2][NW][TM];
    float total[2][NW][2], unit[2][NW][2];
    float dt_plain;  // dt + bias above this is taken as it is
    // What earlier tokens' outputs have to be kept from (see scrub): per head the
    // tile's first step that is not finite (kNoToken: none, kLarge: none, but a
    // large weight), per loading wave whether it loaded an x that is large or not
    // finite, and per column of a wave the first token taken out.  And whether the
    // tile is a gentle one for the head.
    int odd_dt[2][NW], odd_x[NW], gentle[2][NW];
    alignas(16) uint8_t taken[NW][OUT ? 32 : 1];
};
constexpr int kNoToken = TM, kLarge = TM + 1;  // both behind every token

// Column of a unit that row / column l32 of its matrices stands for.
__device__ __forceinline__ int unit_column(int l32) { return 16 * ((l32 >> 2) & 1) + 4 * (l32 >> 3) + (l32 & 3); }

// The state of a unit, [NT tiles][4 i][4 q] with n = 32 tile + 8 i + 4 half + q.
template <int N>
__device__ __forceinline__ void load_state(const void *base, int kind, int64_t at, f32x16_t (&s)[N / 32])
{
#pragma unroll
    for (int nt = 0; nt < N / 32; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kind == kFp32) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(base) + at + 32 * nt + 8 * i);
#pragma unroll
                for (int q = 0; q < 4; ++q) s[nt][4 * i + q] = v[q];
            } else if (kind == kBf16) {
                const u32x2_t v = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(base) + at + 32 * nt + 8 * i);
                s[nt][4 * i] = lo_f32(v[0]);
                s[nt][4 * i + 1] = hi_f32(v[0]);
                s[nt][4 * i + 2] = lo_f32(v[1]);
                s[nt][4 * i + 3] = hi_f32(v[1]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) s[nt][4 * i + q] = 0.0f;
            }
        }
}
template <int N>
__device__ __forceinline__ void store_state(void *base, int kind, int64_t at, const f32x16_t (&s)[N / 32])
{
#pragma unroll
    for (int nt = 0; nt < N / 32; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kind == kFp32)
                *reinterpret_cast<f32x4_t *>(static_cast<float *>(base) + at + 32 * nt + 8 * i) =
                    f32x4_t{s[nt][4 * i], s[nt][4 * i + 1], s[nt][4 * i + 2], s[nt][4 * i + 3]};
            else
                *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(base) + at + 32 * nt + 8 * i) =
                    u32x2_t{pack_bf16x2(s[nt][4 * i], s[nt][4 * i + 1]), pack_bf16x2(s[nt][4 * i + 2], s[nt][4 * i + 3])};
        }
}

// OUT: the pass that writes out (and the final state).  Otherwise the pass
// that forms every segment's own state (from zero) and decay, for all
// segments but a sequence's last; it walks the tiles backwards with weights up
// to the segment's end, so that the accumulators never decay.
template <int N, bool OUT>
__global__ __launch_bounds__(kThreads, 2) void ssm_chunk_kernel(SsmParams p, int units, int ublocks)
{
    constexpr int NT = N / 32, PB = N / 8, PX = NW * 4;  // state tiles; 16-byte pieces of a b and an x row
    // tokens of b (and c) and of x that the threads load at once, and how often
    constexpr int SB = kThreads / PB < TM ? kThreads / PB : TM, kLoadB = TM / SB;
    constexpr int SX = kThreads / PX, kLoadX = TM / SX;
    constexpr int kPitch = Shared<N, OUT>::kPitch;
    constexpr int kStep = OUT ? TM : -TM;
    // With 256 state columns the registers hold no tile in flight.
    constexpr bool kAhead = N <= 128 || !OUT;
    __shared__ __align__(16) Shared<N, OUT> sh;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t gb = static_cast<uint32_t>(p.G) * ublocks, slot = blockIdx.x / gb, in_slot = blockIdx.x - slot * gb;
    const int grp = in_slot / ublocks, ub = in_slot - grp * ublocks;
    const uint32_t seg = static_cast<uint32_t>(p.seg);
    const Tile tile = find_tile(p.seqs, seg, slot);
    const uint32_t t0 = tile.index * seg, left = tile.end - tile.begin - t0;
    const bool last = left <= seg;
    if (!tile.valid || (!OUT && last))
        return;
    const int tokens = static_cast<int>(last ? left : seg);  // of this segment

    const int u0 = ub * NW, u = u0 + wave;  // units within the group
    const bool active = u < units;
    const int per_head = static_cast<int>(p.P / 32);
    const int head0 = u0 / per_head, heads = ((u0 + NW < units ? u0 + NW : units) - 1) / per_head - head0 + 1;
    const int hg = active ? u / per_head : head0, colblk = active ? u - hg * per_head : 0, hs = hg - head0;
    const int h = grp * static_cast<int>(p.H / p.G) + hg, width = static_cast<int>(p.H * p.P);
    const int64_t first = static_cast<int64_t>(tile.begin) + t0;               // the segment's first token in its row
    const int start = OUT ? 0 : (tokens - 1) / TM * TM;  // the first tile walked
    const bool keeps_dt = wave < heads;                  // wave k < heads: works out head k's decays
    const int dh = h - hg + head0 + (keeps_dt ? wave : 0);
    // Places in memory: a base per wave, which moves with the tiles, and 32-bit
    // lane offsets.  Of a tile's b, c and x a wave loads whole rows of 16-byte
    // pieces; of z and out, lane (l32, half) takes 16 columns of token l32.
    const int wb = wave * (64 / PB), wx0 = wave * (64 / PX);  // the first row of either kind
    const char *bp = bytes(p.b + tile.row * p.bb + (first + start + wb) * p.bt + grp * N);
    const char *cp = bytes(p.c + tile.row * p.cb + (first + start + wb) * p.ct + grp * N);
    const char *xp = bytes(p.x + tile.row * p.xb + (first + start + wx0) * p.xt + (grp * units + u0) * 32);
    const char *dp = bytes(p.dt + tile.row * p.db + (first + start) * p.dtt + dh);
    const int wcol = h * static_cast<int>(p.P) + colblk * 32;  // the unit's first output column
    const char *zp = OUT && p.z ? bytes(p.z + tile.row * p.zb + first * p.zt + wcol) : nullptr;
    char *op = reinterpret_cast<char *>(p.out + (tile.row * p.seqs.T + first) * width + wcol);
    // The unit in the states, and in its segment's slab [H][P / 32][4 N / 32][lane][4].
    const int64_t state_at = ((tile.n * p.H + h) * p.P + colblk * 32) * N;
    const int64_t slab_no = p.map.mul * (tile.begin / seg) + p.map.add * tile.n + tile.index;
    float *const slab = p.slabs + ((slab_no * p.H + h) * p.P + colblk * 32) * N;

    // One value a wave each, kept in scalar registers.
    const float rate = of_wave(-expf(p.A_log[dh]) * kLog2eF);
    const float dt_bias = of_wave(p.dt_bias ? p.dt_bias[dh] : 0.0f);
    const float skip = of_wave(OUT && p.D ? p.D[h] : 0.0f);

    f32x16_t s[NT];
    if (OUT && active && !(last && tile.index == 0)) {  // one of several segments
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t *>(slab + (4 * nt + i) * 256 + 4 * lane);
#pragma unroll
                for (int q = 0; q < 4; ++q) s[nt][4 * i + q] = v[q];
            }
    } else {
        load_state<N>(p.init_state, OUT && active ? p.init_kind : kNone,
                      state_at + unit_column(lane & 31) * N + 4 * (lane >> 5), s);
    }
    // Where the unit's final state goes, if it does; bit 0: in bf16.
    char *final_at = nullptr;
    if (OUT && last && p.final_state)
        final_at = static_cast<char *>(p.final_state) + (p.final_kind == kFp32 ? 4 * state_at : 2 * state_at + 1);
    if (OUT && tid < 256) {
        // c b^T is 0 above the diagonal; a block's upper right 16 x 16 is never
        // written again: t < 16, s >= 16 are slots e with e % 4 >= 2
        const int part = tid >> 7, blk = (tid >> 6) & 1, j = (tid >> 5) & 1, hf = (tid >> 4) & 1;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e & 2)
                sh.cb[blk][part][j][hf][tid & 15][e] = 0;
    }

    u32x4_t rb[kLoadB], rc[OUT ? kLoadB : 1], rx[kLoadX] = {};
    uint32_t rdt = 0;
    float after = 0.0f;  // sum of a over the tiles after this one (!OUT; this wave's dt head)
    // Loads the tile from token tt on and moves on to the next.
    const auto fetch = [&](int tt) {
        const int ln = here(lane), bt0 = wb + ln / PB, xt0 = wx0 + ln / PX;
        const uint32_t b_off = 2 * (ln / PB * static_cast<uint32_t>(p.bt) + ln % PB * 8);
        const uint32_t c_off = 2 * (ln / PB * static_cast<uint32_t>(p.ct) + ln % PB * 8);
        const uint32_t x_off = 2 * (ln / PX * static_cast<uint32_t>(p.xt) + ln % PX * 8);
        const bool x_here = ln % PX * 8 < (units - u0) * 32;  // a column of a unit that exists
        const char *bq = bp, *cq = cp, *xq = xp;
        if (tt + TM <= tokens) {
#pragma unroll
            for (int k = 0; k < kLoadB; ++k) {
                if (SB * PB == kThreads || bt0 < SB) {
                    rb[k] = *reinterpret_cast<const u32x4_a2 *>(bq + b_off);
                    if constexpr (OUT)
                        rc[k] = *reinterpret_cast<const u32x4_a2 *>(cq + c_off);
                }
                bq += 2 * SB * p.bt;
                cq += 2 * SB * p.ct;
            }
#pragma unroll
            for (int k = 0; k < kLoadX; ++k) {
                if (x_here)
                    rx[k] = *reinterpret_cast<const u32x4_a2 *>(xq + x_off);
                xq += 2 * SX * p.xt;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kLoadB; ++k) {
                const bool ok = bt0 < SB && tt + bt0 + k * SB < tokens;
                rb[k] = ok ? *reinterpret_cast<const u32x4_a2 *>(bq + b_off) : u32x4_t{0, 0, 0, 0};
                if constexpr (OUT)
                    rc[k] = ok ? *reinterpret_cast<const u32x4_a2 *>(cq + c_off) : u32x4_t{0, 0, 0, 0};
                bq += 2 * SB * p.bt;
                cq += 2 * SB * p.ct;
            }
#pragma unroll
            for (int k = 0; k < kLoadX; ++k) {
                const bool ok = x_here && tt + xt0 + k * SX < tokens;
                rx[k] = ok ? *reinterpret_cast<const u32x4_a2 *>(xq + x_off) : u32x4_t{0, 0, 0, 0};
                xq += 2 * SX * p.xt;
            }
        }
        bp += 2 * kStep * p.bt;
        cp += 2 * kStep * p.ct;
        xp += 2 * kStep * p.xt;
    };
    // dt of the tile from token tt on, loaded one step ahead of its use
    const auto fetch_dt = [&](int tt) {
        const int ln = here(lane);
        rdt = 0;
        if (keeps_dt && tt >= 0 && tt + ln < tokens)
            rdt = *reinterpret_cast<const uint16_t *>(dp + 2 * ln * p.dtt);
        dp += 2 * kStep * p.dtt;
    };
    // What the loaded dt of the tile from token tt on comes to, into its half of the buffers.
    const auto step_dt = [&](int tt, float plain) {
        const int ln = here(lane), buf = (tt / TM) & 1;
        const float raw = bf16_to_f32(static_cast<uint16_t>(rdt)) + dt_bias;
        const bool inside = tt + ln < tokens;  // behind the end nothing decays, however strong the rate
        float dt = inside ? softplus_f32(raw, plain) : 0.0f;
        const float log_keep = inside ? rate * dt : 0.0f;
        // Not a number, or a growth beyond fp32: as a step that is not finite, and
        // in the sums as the strongest decay.
        const bool keeps = log_keep < 128.0f;
        const float a = keeps ? fmaxf(log_keep, -160.0f) : -160.0f;
        dt = keeps ? dt : __builtin_nanf("");
        float r = after32(a, ln);
        uint64_t odd = 0;
        if constexpr (OUT) {
            const bool finite = fabsf(dt) < __builtin_inff();
            odd = __ballot(!finite);
            dt = finite ? dt : 0.0f;
            const float abs_sum = prefix32(fabsf(a));
            const float s0 = read_lane(abs_sum, 31), s1 = read_lane(abs_sum, 63);
            // 2^e <= sum < 2^(e + 1): a unit of 2^(e - 29)
            const uint32_t e = __float_as_uint(fmaxf(ln < 32 ? s0 : s1, 0x1p-60f)) & 0x7f800000u;
            const float unit = __uint_as_float(e - (29u << 23));
            const int g = prefix32(static_cast<int>(rintf(a * __uint_as_float((254u << 23) - e + (29u << 23)))));
            sh.g[buf][wave][ln] = g;
            sh.d[buf][wave][ln] = dt;
            const float total = unit * static_cast<float>(g);
            if ((ln & 31) == 31) {
                sh.unit[buf][wave][ln >> 5] = unit;
                sh.total[buf][wave][ln >> 5] = total;
            }
            // a gentle tile weighs its first block up to the tile's end
            const float b1 = read_lane(r + a, 32), both = read_lane(total, 31) + read_lane(total, 63);
            const float to_end = r + (ln < 32 ? b1 : 0.0f);
            const bool gentle = kAhead && !__any(fabsf(to_end) > -kSteep || both < kSteep);
            r = gentle ? to_end : r;
            if (ln == 0)
                sh.gentle[buf][wave] = gentle;
        } else {
            // from the block's end to the segment's
            const float b0 = read_lane(r + a, 0), b1 = read_lane(r + a, 32);
            if (ln == 0) {
                sh.total[buf][wave][0] = b1 + after;
                sh.total[buf][wave][1] = after;
            }
            r += ln < 32 ? b1 + after : after;
            after += b0 + b1;
        }
        const float w = dt * exp2_f32(r);
        sh.w[buf][wave][ln] = w;
        if constexpr (OUT) {
            const bool large = __any(!(fabsf(w) < kLargeWeight));
            if (ln == 0)
                sh.odd_dt[buf][wave] = odd ? __builtin_ctzll(odd) : large ? kLarge : kNoToken;
        }
    };
    const auto put = [](uint16_t *dst, u32x4_t v) {  // rows are 8-byte aligned
        *reinterpret_cast<u32x2_t *>(dst) = u32x2_t{v[0], v[1]};
        *reinterpret_cast<u32x2_t *>(dst + 4) = u32x2_t{v[2], v[3]};
    };

    if (tokens > 0) {
        fetch_dt(start);
        if (kAhead)
            fetch(start);
        const float plain = dt_plain_above(p.softplus);
        if (tid == 0)
            sh.dt_plain = plain;
        if (keeps_dt)
            step_dt(start, plain);
        fetch_dt(start + kStep);
    }
    // The tiles of c b^T this wave forms: two for a wave without a head, the
    // rest for the others.
    const int spare = NW - heads, share = 2 * spare < 10 ? 2 * spare : 10;
    int ids = 0xffff;
    if (OUT) {
        for (int id = 0; id < 10; ++id)
            if (wave == (id < share ? heads + id % spare : (id - share) % heads))
                ids = (ids << 8 | id) & 0xffff;
    }

    for (int tt = start; OUT ? tt < tokens : tt >= 0; tt += kStep) {
        if (tokens == 0)
            break;
        if (!kAhead)
            fetch(tt);
        {
            const int ln = here(lane), bt0 = wb + ln / PB, bc0 = ln % PB * 8;
#pragma unroll
            for (int k = 0; k < kLoadB; ++k) {
                if (SB * PB == kThreads || bt0 < SB) {
                    put(&sh.b[bt0 + k * SB][bc0], rb[k]);
                    if constexpr (OUT)
                        put(&sh.c[bt0 + k * SB][bc0], rc[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < kLoadX; ++k) put(&sh.x[wx0 + ln / PX + k * SX][ln % PX * 8], rx[k]);
            if constexpr (OUT) {
                // squares: not finite once an x is not, or is 2^64 or more
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kLoadX; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum = dot2_bf16(rx[k][i], rx[k][i], sum);
                const bool odd = __any(!(fabsf(sum) < __builtin_inff()));
                if (ln == 0)
                    sh.odd_x[wave] = odd;
            }
        }
        lds_barrier();
        const int buf = (tt / TM) & 1;
        const bool more = OUT ? tt + TM < tokens : tt > 0;
        // The next tile's dt, and this one's c b^T, a wave each where it can be.
        if (more) {
            if (keeps_dt)
                step_dt(tt + kStep, sh.dt_plain);
            fetch_dt(tt + 2 * kStep);
        }
        // the tile after it, in flight from here on
        if (kAhead && more)
            fetch(tt + kStep);
        if constexpr (OUT) {
            const int ln = here(lane), l16 = ln & 15, g4 = ln >> 4;
            for (int k = 0; k < 2; ++k) {
                const int id = (ids >> (8 * k)) & 0xff;
                if (id == 0xff)
                    break;
                const int ti = id < 1 ? 0 : (id < 3 ? 1 : (id < 6 ? 2 : 3)), si = id - ti * (ti + 1) / 2;
                f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint16_t *pb = &sh.b[16 * si + l16][32 * n + 8 * g4];
                    const uint16_t *pc = &sh.c[16 * ti + l16][32 * n + 8 * g4];
                    const bf16x8_t vb = cat8(*reinterpret_cast<const u32x2_t *>(pb), *reinterpret_cast<const u32x2_t *>(pb + 4));
                    const bf16x8_t vc = cat8(*reinterpret_cast<const u32x2_t *>(pc), *reinterpret_cast<const u32x2_t *>(pc + 4));
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, vc, acc, 0, 0, 0);
                }
                // the lane's t = 16 ti + l16, s = 16 si + 4 g4 + r
                const int blk = (ti >> 1) == (si >> 1) ? ti >> 1 : 2;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = si == ti && 4 * g4 + r > l16 ? 0.0f : acc[r];
                    const uint32_t hi = pack_bf16x2(v, 0.0f), lo = pack_bf16x2(v - lo_f32(hi), 0.0f);
                    const int e = 2 * (si & 1) + (g4 >> 1) + 4 * (r & 1);
                    sh.cb[blk][0][r >> 1][g4 & 1][16 * (ti & 1) + l16][e] = static_cast<uint16_t>(hi);
                    sh.cb[blk][1][r >> 1][g4 & 1][16 * (ti & 1) + l16][e] = static_cast<uint16_t>(lo);
                }
            }
            lds_barrier();
        }
        u32x4_t rz[2][2];  // z of the lane's token of either block
        if (OUT && zp && active) {
            const int ln = here(lane), l32 = ln & 31;
            const uint32_t z_off = 2 * (l32 * static_cast<uint32_t>(p.zt) + 16 * (ln >> 5));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (tt + CH * q + l32 < tokens) {
                    rz[q][0] = *reinterpret_cast<const u32x4_a2 *>(zp + z_off);
                    rz[q][1] = *reinterpret_cast<const u32x4_a2 *>(zp + 16 + z_off);
                }
                zp += 2 * CH * p.zt;
            }
        }
        if (active) {
            // Where a SIMD's waves have got to: the one behind goes first, so
            // that neither runs alone at the end.
            __builtin_amdgcn_s_setprio(3);
            const int ln = here(lane), l32 = ln & 31, half = ln >> 5, l16 = ln & 15, odd = (ln >> 4) & 1;
            // of the transposing reads of b and x
            const uint32_t b_tr = lds_addr(&sh.b[4 * half + 8 * (l16 >> 2)][16 * odd + 4 * (l16 & 3)]);
            const int kappa = 4 * odd + (l16 & 3);
            const uint32_t x_tr = lds_addr(&sh.x[4 * half + 8 * (l16 >> 2)][wave * 32 + 16 * (kappa & 1) + 4 * (kappa >> 1)]);
            // x_s of a block, column l32, tokens in contraction order
            const auto load_x = [&](int q, int j) {
                const uint32_t a = x_tr + 2 * kXPitch * (CH * q + 2 * j);
                return cat8(lds_tr(a), lds_tr(a + 2 * kXPitch));
            };
            // w_s x_s in two or three parts, or (1) the third that two leave out
            const auto weighted = [&](auto parts, int q, bf16x8_t(&wx)[2][3]) {
                float w[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4_t v = *reinterpret_cast<const f32x4_t *>(&sh.w[buf][hs][CH * q + 8 * i + 4 * half]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[i][e] = v[e];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[8];
                    unpack8(__builtin_bit_cast(u32x4_t, load_x(q, j)), v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= w[e & 3][2 * j + (e >> 2)];
                    if constexpr (parts() == 1)
                        wx[j][2] = rest8(v);
                    else
                        split8<parts()>(v, wx[j]);
                }
            };
            // S += parts k0 .. k1 - 1 of sum_s w_s x_s b_s^T over block q
            const auto update = [&](int q, auto k0, auto k1, int nt, const bf16x8_t(&wx)[2][3]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t a = b_tr + 2 * kPitch * (CH * q + 2 * j) + 64 * nt;
                    const bf16x8_t vb = cat8(lds_tr(a), lds_tr(a + 2 * kPitch));
#pragma unroll
                    for (int k = k0(); k < k1(); ++k) s[nt] = mfma(vb, wx[j][k], s[nt]);
                }
                if constexpr (N > 128)
                    fence();  // registers are short: no operand is read early
            };
            // The third part by itself: y's sums hold registers that it would need.
            const auto refine = [&](int q) {
                bf16x8_t wx[2][3];
                weighted(Int<1>(), q, wx);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) update(q, Int<2>(), Int<3>(), nt, wx);
            };
            const int odd_dt = OUT ? __builtin_amdgcn_readfirstlane(sh.odd_dt[buf][hs]) : kNoToken;
            const bool suspect = OUT && (odd_dt != kNoToken || __any(sh.odd_x[ln & (NW - 1)]));
            // A product of 0 (in c b^T, M) and what is not finite is NaN, and would
            // take a token into the outputs before it.  So an x whose product with
            // its weight is not finite leaves its column (0 in its place), as a step
            // that is not finite has left the weights, and the outputs from its token
            // on and the state are made NaN (spoil, finish).
            const auto scrub = [&]() {
                const int t = here(ln);
                int mine = kNoToken;  // of column t & 31
                const float w = sh.w[buf][hs][t];
#pragma unroll 1
                for (int c = 0; c < 32; ++c) {
                    uint16_t *x = &sh.x[t][wave * 32 + c];
                    const bool out = !(fabsf(w * bf16_to_f32(*x)) < 0x1.ffp127f);  // as bf16 infinite from there on
                    if (out)
                        *x = 0;
                    const uint64_t tokens_out = __ballot(out);
                    mine = tokens_out && (t & 31) == c ? __builtin_ctzll(tokens_out) : mine;
                }
                if (t < 32)
                    sh.taken[wave][t] = static_cast<uint8_t>(mine < odd_dt ? mine : odd_dt);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            };
            const auto spoil = [&]() {
                const bool gone = sh.taken[wave][unit_column(here(l32))] < kNoToken;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[nt][r] = gone ? __builtin_nanf("") : s[nt][r];
            };
            if constexpr (OUT) {
                if (suspect)
                    scrub();
            }
            if constexpr (!OUT) {
#pragma unroll 1
                for (int q = 1; q >= 0; --q) {
                    const float rest = read_lane(sh.total[buf][hs][q], 0);  // from the block's end to the segment's
                    if (rest < kNothing)
                        break;
                    bf16x8_t wx[2][3];
                    weighted(Int<3>(), q, wx);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) update(q, Int<0>(), Int<3>(), nt, wx);
                }
            } else {
                const bool updates = more || final_at;
                const float total0 = read_lane(sh.total[buf][hs][0], 0), total1 = read_lane(sh.total[buf][hs][1], 0);
                const bool gentle = kAhead && __builtin_amdgcn_readfirstlane(sh.gentle[buf][hs]);  // never with 256 state columns
                f32x16_t y[2];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int r = 0; r < 16; ++r) y[q][r] = 0.0f;
                // y += S c_t of both blocks
                const auto add_carried = [&]() {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (!kAhead)
                            fence();
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = s[nt][8 * j + e];
                            bf16x8_t parts[2];
                            split8<2>(v, parts);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint16_t *pc = &sh.c[CH * q + l32][32 * nt + 16 * j + 4 * half];
                                const bf16x8_t vc = cat8(*reinterpret_cast<const u32x2_t *>(pc), *reinterpret_cast<const u32x2_t *>(pc + 8));
                                y[q] = mfma(parts[0], vc, y[q]);
                                y[q] = mfma(parts[1], vc, y[q]);
                            }
                        }
                    }
                };
                // y[q] += sum_s (c_t . b_s) w_s x_s over the tokens s that c b^T number blk has
                const auto add_weighted = [&](int q, int blk, const bf16x8_t(&wx)[2][3]) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bf16x8_t hi = *reinterpret_cast<const bf16x8_t *>(sh.cb[blk][0][j][half][l32]);
                        const bf16x8_t lo = *reinterpret_cast<const bf16x8_t *>(sh.cb[blk][1][j][half][l32]);
                        y[q] = mfma(wx[j][0], hi, y[q]);
                        y[q] = mfma(wx[j][1], hi, y[q]);
                        y[q] = mfma(wx[j][0], lo, y[q]);
                    }
                };
                const auto decay_state = [&](float keep) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[nt][r] *= keep;
                };
                const auto log_to = [&](int q) {  // G of the lane's token of block q
                    return read_lane(sh.unit[buf][hs][q], 0) * static_cast<float>(sh.g[buf][hs][CH * q + l32]);
                };
                // out of block q from f y[q]
                const auto finish = [&](int q, float f) {
                    if (tt + CH * q + l32 < tokens) {
                        float o[16];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint16_t *px = &sh.x[CH * q + l32][wave * 32 + 16 * half + 8 * k];
                            const u32x2_t x0 = *reinterpret_cast<const u32x2_t *>(px), x1 = *reinterpret_cast<const u32x2_t *>(px + 4);
                            unpack8(u32x4_t{x0[0], x0[1], x1[0], x1[1]}, o + 8 * k);
                        }
#pragma unroll
                        for (int r = 0; r < 16; ++r) o[r] = fmaf(f, y[q][r], skip * o[r]);
                        if (zp) {
                            float z[16];
                            unpack8(rz[q][0], z);
                            unpack8(rz[q][1], z + 8);
#pragma unroll
                            for (int r = 0; r < 16; ++r) o[r] *= silu_f32(z[r]);
                        }
                        if (suspect) {
                            const u32x4_t from = *reinterpret_cast<const u32x4_t *>(&sh.taken[wave][here(16 * half)]);
                            const uint32_t at = here(l32) + CH * q;
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                o[r] = (from[r / 4] >> (8 * (r & 3)) & 0xff) <= at ? __builtin_nanf("") : o[r];
                        }
                        const uint32_t o_off = 2 * (l32 * static_cast<uint32_t>(width) + 16 * half);
                        *reinterpret_cast<u32x4_t *>(op + o_off) = pack8(o);
                        *reinterpret_cast<u32x4_t *>(op + 16 + o_off) = pack8(o + 8);
                    }
                    op += 2 * CH * width;
                };
                if (gentle) {
                    decay_state(exp2_f32(total0 + total1));
                    add_carried();
                    __builtin_amdgcn_s_setprio(2);
                    bf16x8_t wx[2][3];
                    weighted(Int<2>(), 0, wx);
                    add_weighted(0, 0, wx);
                    add_weighted(1, 2, wx);
                    if (updates) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) update(0, Int<0>(), Int<2>(), nt, wx);
                    }
                    finish(0, exp2_f32(log_to(0) - (total0 + total1)));
                    __builtin_amdgcn_s_setprio(1);
                    weighted(Int<3>(), 1, wx);
                    add_weighted(1, 1, wx);
                    if (updates) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) update(1, Int<0>(), Int<3>(), nt, wx);
                        refine(0);
                    }
                    finish(1, exp2_f32(log_to(1) - total1));
                } else {
                    add_carried();
                    __builtin_amdgcn_s_setprio(2);
                    const float keep0 = exp2_f32(total0);
#pragma unroll
                    for (int r = 0; r < 16; ++r) y[1][r] *= keep0;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float total = q ? total1 : total0, log_t = log_to(q);
                        bf16x8_t wx[2][3];
                        weighted(Int<2>(), q, wx);
                        if (q == 0)
                            add_weighted(1, 2, wx);
                        if (updates) {
                            decay_state(exp2_f32(total));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) update(q, Int<0>(), Int<2>(), nt, wx);
                            refine(q);
                        }
                        // M[t, s] = (c_t . b_s) dt_s 2^(G_t - G_s) over the block's own tokens
                        const float f = exp2_f32(log_t);
#pragma unroll
                        for (int r = 0; r < 16; ++r) y[q][r] *= f;
                        const float unit = read_lane(sh.unit[buf][hs][q], 0);
                        const int gt = sh.g[buf][hs][CH * q + l32];
#pragma unroll 1
                        for (int j = 0; j < 2; ++j) {
                            const u32x4_t hi = *reinterpret_cast<const u32x4_t *>(sh.cb[q][0][j][half][l32]);
                            const u32x4_t lo = *reinterpret_cast<const u32x4_t *>(sh.cb[q][1][j][half][l32]);
                            float m[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                // c b^T is 0 for s > t, where the factor only has to stay finite
                                const int at = CH * q + 8 * (e & 3) + 4 * half + 2 * j + (e >> 2);
                                const float span = fminf(unit * static_cast<float>(gt - sh.g[buf][hs][at]), 120.0f);
                                const float cb = e & 1 ? hi_f32(hi[e / 2]) + hi_f32(lo[e / 2]) : lo_f32(hi[e / 2]) + lo_f32(lo[e / 2]);
                                m[e] = cb * sh.d[buf][hs][at] * exp2_f32(span);
                            }
                            bf16x8_t parts[2];
                            split8<2>(m, parts);
                            const bf16x8_t xa = load_x(q, j);
                            y[q] = mfma(xa, parts[0], y[q]);
                            y[q] = mfma(xa, parts[1], y[q]);
                        }
                        finish(q, 1.0f);
                    }
                }
                if (suspect)
                    spoil();
            }
            __builtin_amdgcn_s_setprio(3);
        }
        lds_barrier();
        if constexpr (!OUT) {
            // nothing earlier reaches the segment's end: the weights are 0
            bool nothing = true;
            for (int k = 0; k < heads; ++k) nothing &= read_lane(sh.total[buf][k][0], 0) < kNothing;
            if (nothing)
                break;
        }
    }

    if constexpr (OUT) {
        if (active && final_at) {
            const int ln = here(lane);
            const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(final_at) & 1);
            store_state<N>(final_at - odd, odd ? kBf16 : kFp32, unit_column(ln & 31) * N + 4 * (ln >> 5), s);
        }
    } else {
        if (active) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<f32x4_t *>(slab + (4 * nt + i) * 256 + 4 * lane) =
                        f32x4_t{s[nt][4 * i], s[nt][4 * i + 1], s[nt][4 * i + 2], s[nt][4 * i + 3]};
        }
        // Several workgroups may hold columns of one head, and their sums may differ
        // below kNothing, where each stops: the one with the first column writes.
        if (keeps_dt && lane == 0 && (wave > 0 || head0 * per_head == u0))
            p.logs[slab_no * p.H + dh] = after;
    }
}

// The states in front of the segments, in order: start_0 = the initial state,
// start_(k+1) = 2^(log decay of k) start_k + own state of k, each over its
// segment's slab.  (The first one too: the output pass may write the final
// state over the initial one.)  Sequences of one segment are left to the output
// pass.  A thread carries four elements of one (sequence, head).
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void ssm_join_kernel(SsmParams p, int64_t quads)
{
    const uint32_t per = (static_cast<uint32_t>(quads) + kJoinThreads - 1) / kJoinThreads, chain = blockIdx.x / per;
    const uint32_t q = (blockIdx.x - chain * per) * kJoinThreads + threadIdx.x;  // quad within the head's slab
    const uint32_t heads = static_cast<uint32_t>(p.H), seg = static_cast<uint32_t>(p.seg);
    const int64_t n = chain / heads, h = chain - static_cast<uint32_t>(n) * heads;
    uint32_t begin = 0, end = static_cast<uint32_t>(p.seqs.T);
    if (p.seqs.cu) {
        begin = clamp_offset(p.seqs, n);
        end = clamp_offset(p.seqs, n + 1);
    }
    const uint32_t count = end > begin ? (end - begin - 1) / seg + 1 : 1;
    if (q >= quads || count == 1)
        return;
    f32x4_t run = {0, 0, 0, 0};
    if (p.init_kind != kNone) {
        // quad q of the slab: unit, tile and i, lane
        const int64_t unit = q / (p.N * 8), in = q - unit * (p.N * 8);
        const int ti = static_cast<int>(in >> 6), lane = static_cast<int>(in & 63);
        const int64_t at = ((n * p.H + h) * p.P + unit * 32 + unit_column(lane & 31)) * p.N + 8 * ti + 4 * (lane >> 5);
        if (p.init_kind == kFp32) {
            run = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p.init_state) + at);
        } else {
            const u32x2_t v = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(p.init_state) + at);
            run = f32x4_t{lo_f32(v[0]), hi_f32(v[0]), lo_f32(v[1]), hi_f32(v[1])};
        }
    }
    const int64_t step = p.H * p.P * p.N;
    const int64_t slab_no = p.map.mul * (begin / seg) + p.map.add * n;
    float *slab = p.slabs + (slab_no * p.H + h) * p.P * p.N + 4 * q;
    const float *logs = p.logs + slab_no * p.H + h;
    // eight segments' loads at once: a store of this loop could be what the
    // next load reads, as far as the compiler knows
    constexpr uint32_t kAhead = 8;
    for (uint32_t k0 = 0; k0 + 1 < count; k0 += kAhead) {
        f32x4_t own[kAhead];
        float keep[kAhead];
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i)
            if (k0 + i + 1 < count) {
                own[i] = *reinterpret_cast<const f32x4_t *>(slab + (k0 + i) * step);
                keep[i] = logs[(k0 + i) * p.H];
            }
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i)
            if (k0 + i + 1 < count) {
                *reinterpret_cast<f32x4_t *>(slab + (k0 + i) * step) = run;
                const float f = exp2_f32(keep[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) run[e] = fmaf(f, run[e], own[i][e]);
            }
    }
    *reinterpret_cast<f32x4_t *>(slab + (count - 1) * step) = run;
}

template <int N>
hipError_t launch(const SsmParams &p, hipStream_t stream)
{
    const int units = static_cast<int>(p.H / p.G * (p.P / 32)), ublocks = (units + NW - 1) / NW;
    const int64_t blocks = tile_slots(p.seqs, p.seg) * p.G * ublocks;
    const int64_t quads = p.P * N / 4, join = p.seqs.N * p.H * ((quads + kJoinThreads - 1) / kJoinThreads);
    if (!grid_fits(blocks, kThreads) || (p.slabs && !grid_fits(join, kJoinThreads)))
        return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (p.slabs) {
        ssm_chunk_kernel<N, false><<<grid, dim3(kThreads), 0, stream>>>(p, units, ublocks);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        ssm_join_kernel<<<dim3(static_cast<uint32_t>(join)), dim3(kJoinThreads), 0, stream>>>(p, quads);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    ssm_chunk_kernel<N, true><<<grid, dim3(kThreads), 0, stream>>>(p, units, ublocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_chunk(const SsmParams &p, hipStream_t stream)
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
