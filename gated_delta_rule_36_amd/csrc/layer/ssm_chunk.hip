// The selective state space scan in chunks of 32 tokens on matrix
// instructions.  Per head, with a_t = -e^A_log log2(e) dt_t, G_t the sum of a
// over the chunk up to and with token t, R_t the sum over the tokens after t
// and S the state [P, N] in front of the chunk:
//   M[t,s] = (c_t . b_s) dt_s 2^(G_t - G_s)  (s <= t),  M[t,t] += D
//   y_t    = 2^(G_t) S c_t + sum_s M[t,s] x_s,  out_t = y_t silu(z_t)
//   S     <- 2^(G_last) S + sum_s (dt_s 2^(R_s) x_s) b_s^T
// No exponent is positive, so nothing overflows however strong the decay.  A
// difference of G loses what a strong decay in the same chunk rounds away, so
// G is held in fixed point: 32-bit integers in a unit of 2^-29 .. 2^-30 of the
// chunk's sum of |a|, whose sums and differences are exact.  Decays below
// 2^-160 count as that (both are 0 in fp32), so a unit is at most 2^-17.  R is
// summed in fp32 from the chunk's end, so that the weights of the newest
// tokens, which make up most of the state, are the most exact.
//
// One wave owns a unit: 32 of a head's P columns, with the fp32 state [32, N]
// in accumulators for a whole segment of the sequence.  A workgroup of eight
// waves takes eight consecutive units of one group (P = 64: four heads), which
// share b and c.  Tiles of 64 tokens (two chunks) of b, c and x go through
// registers into LDS, the next tile's loads in flight while this one is
// computed; the products c b^T are formed once per workgroup, one 16 x 16 tile
// a wave.  x is read from memory once per pass, 64 bytes a token and unit.
//
// Operands.  v_mfma_f32_32x32x16_bf16 contracts 16 slots; lane (l32, half)
// holds slots 8 half .. 8 half + 7 of row / column l32, and accumulator
// register r = 4 i + q is row 8 i + 4 half + q.  Which contraction index a
// slot stands for is free as long as both operands agree:
//   over n:  slot e of step (tile, j) is n = 32 tile + 16 j + 8 (e / 4) + 4 half + e % 4,
//            so a state accumulator is the operand as it stands;
//   over s:  slot e of step j is s = 8 (e % 4) + 4 half + 2 j + e / 4, so M as
//            the product c b^T leaves it is the operand, and the four tokens a
//            transposing LDS read takes are 8 rows apart, which with rows of
//            2 mod 16 dwords puts them in distinct banks.
// Row / column l32 of the unit stands for column p = 16 ((l32 >> 2) & 1) +
// 4 (l32 >> 3) + l32 % 4, so that a lane ends with 16 adjacent columns of its
// token's output.
//
// x, b and c are bf16 and enter as they are.  M, the state and the weighted x
// are fp32 and enter as two bf16 parts (the value rounded, and the rest
// rounded: good to 2^-16 of itself), so the state keeps fp32's accuracy to
// better than 2^-18 over its norm and out is good to its one final rounding.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int CH = static_cast<int>(kSsmChunk);
constexpr int TM = 2 * CH;  // tokens a tile
constexpr int NW = 8;       // waves, units a workgroup
constexpr int kThreads = 64 * NW;
constexpr int kXPitch = NW * 32 + 4;  // bf16 elements of an x row in LDS

typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ uint32_t lds_addr(const void *p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8 *)p));
}
// Transposing LDS read: within each 16-lane row, lane L points at four bf16
// X[L][0..3]; lane i receives X[4 r + i / 4][i % 4] for r = 0..3.
__device__ __forceinline__ u32x2_t lds_tr(uint32_t a)
{
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                           (__attribute__((address_space(3))) s16x4_t *)(uintptr_t)a));
}
__device__ __forceinline__ bf16x8_t cat8(u32x2_t a, u32x2_t b)
{
    return __builtin_bit_cast(bf16x8_t, u32x4_t{a[0], a[1], b[0], b[1]});
}
__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// Workgroup barrier that orders LDS only: loads to registers stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// v = hi + lo, each rounded to bf16.
__device__ __forceinline__ void split8(const float v[8], bf16x8_t *hi, bf16x8_t *lo)
{
    u32x4_t h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        l[i] = pack_bf16x2(v[2 * i] - lo_f32(h[i]), v[2 * i + 1] - hi_f32(h[i]));
    }
    *hi = __builtin_bit_cast(bf16x8_t, h);
    *lo = __builtin_bit_cast(bf16x8_t, l);
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

__device__ __forceinline__ float softplus_f32(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

template <int N, bool OUT>
struct Shared {
    static constexpr int kPitch = N + 4;
    uint16_t b[TM][kPitch];
    uint16_t c[OUT ? TM : 1][kPitch];
    uint16_t x[TM][kXPitch];
    float cb[OUT ? TM / CH : 1][CH][CH + 4];  // [t][s] = c_t . b_s of a chunk
    // per wave and token: G in its chunk's units, dt, dt 2^R
    int g[NW][TM];
    float d[NW][TM], w[NW][TM];
};

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
// segments but a sequence's last.
template <int N, bool OUT>
__global__ __launch_bounds__(kThreads, 2) void ssm_chunk_kernel(SsmParams p, int units, int ublocks)
{
    constexpr int NT = N / 32, PB = N / 8;                 // state tiles; 16-byte pieces of a b row
    // tokens of b (and c) and of x that the threads load at once, and how often
    constexpr int SB = kThreads / PB < TM ? kThreads / PB : TM, kLoadB = TM / SB;
    constexpr int SX = kThreads / (NW * 4), kLoadX = TM / SX;
    constexpr int kPitch = Shared<N, OUT>::kPitch;
    __shared__ __align__(16) Shared<N, OUT> sh;

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, half = lane >> 5, l16 = lane & 15, odd = (lane >> 4) & 1;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t gb = p.G * ublocks;
    const int64_t slot = blockIdx.x / gb;
    const int rest = static_cast<int>(blockIdx.x - slot * gb), grp = rest / ublocks, ub = rest - grp * ublocks;
    const Tile tile = find_tile(p.seqs, p.seg, slot);
    const int64_t t0 = tile.index * p.seg, left = tile.end - tile.begin - t0;
    const bool last = left <= p.seg;
    if (!tile.valid || (!OUT && last))
        return;
    const int tokens = static_cast<int>(last ? left : p.seg);  // of this segment

    const int u = ub * NW + wave;  // unit within the group
    const bool active = u < units;
    const int per_head = static_cast<int>(p.P / 32);
    const int hg = (active ? u : 0) / per_head, colblk = (active ? u : 0) - hg * per_head;
    const int64_t h = grp * (p.H / p.G) + hg;
    const int64_t first = tile.begin + t0;                  // the segment's first token in its row
    const int64_t col = h * p.P + colblk * 32 + 16 * half;  // the lane's first output column
    // This thread's places in memory: piece 0 of a tile's b, c and x, the
    // token `lane` of dt, the token l32 of z and out; they advance by chunks
    // or tiles.
    const int bt0 = tid / PB, bc0 = tid % PB * 8, xt0 = tid / (NW * 4), xc0 = tid % (NW * 4) * 8;
    const uint16_t *bp = p.b + tile.row * p.bb + (first + bt0) * p.bt + static_cast<int64_t>(grp) * N + bc0;
    const uint16_t *cp = p.c + tile.row * p.cb + (first + bt0) * p.ct + static_cast<int64_t>(grp) * N + bc0;
    const uint16_t *xp = p.x + tile.row * p.xb + (first + xt0) * p.xt + (static_cast<int64_t>(grp) * units + ub * NW) * 32 + xc0;
    const uint16_t *dp = p.dt + tile.row * p.db + (first + lane) * p.dtt + h;
    const uint16_t *zp = OUT && p.z ? p.z + tile.row * p.zb + (first + l32) * p.zt + col : nullptr;
    uint16_t *op = p.out + (tile.row * p.seqs.T + first + l32) * p.H * p.P + col;
    const int64_t state_at = ((tile.n * p.H + h) * p.P + colblk * 32 + unit_column(l32)) * N + 4 * half;
    float *slab = p.slabs + ((slot * p.H + h) * p.P + colblk * 32) * N + 4 * lane;  // [NT * 4][lane][4]

    const float rate = -expf(p.A_log[h]) * kLog2eF;
    const float dt_bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = OUT && p.D ? p.D[h] : 0.0f;

    f32x16_t s[NT];
    if (OUT && active && p.slabs) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t *>(slab + (4 * nt + i) * 256);
#pragma unroll
                for (int q = 0; q < 4; ++q) s[nt][4 * i + q] = v[q];
            }
    } else {
        load_state<N>(p.init_state, OUT && active ? p.init_kind : kNone, state_at, s);
    }
    float log_sum = 0.0f;
    float diag[16];  // D where row s = 8 i + 4 half + q is the lane's own token
#pragma unroll
    for (int r = 0; r < 16; ++r) diag[r] = 8 * (r >> 2) + 4 * half + (r & 3) == l32 ? skip : 0.0f;

    u32x4_t rb[kLoadB], rc[OUT ? kLoadB : 1], rx[kLoadX];
    uint32_t rdt = 0;
    const bool x_here = xc0 < units * 32 - ub * NW * 32;  // a column of a unit that exists
    // Loads the tile from token tt on (of which `tokens - tt` exist) and moves on to the next.
    const auto fetch = [&](int tt) {
#pragma unroll
        for (int k = 0; k < kLoadB; ++k) {
            const bool ok = bt0 < SB && tt + bt0 + k * SB < tokens;
            rb[k] = ok ? *reinterpret_cast<const u32x4_a2 *>(bp) : u32x4_t{0, 0, 0, 0};
            bp += SB * p.bt;
            if constexpr (OUT) {
                rc[k] = ok ? *reinterpret_cast<const u32x4_a2 *>(cp) : u32x4_t{0, 0, 0, 0};
                cp += SB * p.ct;
            }
        }
#pragma unroll
        for (int k = 0; k < kLoadX; ++k) {
            const bool ok = x_here && tt + xt0 + k * SX < tokens;
            rx[k] = ok ? *reinterpret_cast<const u32x4_a2 *>(xp) : u32x4_t{0, 0, 0, 0};
            xp += SX * p.xt;
        }
        rdt = tt + lane < tokens ? *dp : 0;
        dp += TM * p.dtt;
    };
    const auto put = [](uint16_t *dst, u32x4_t v) {  // rows are 8-byte aligned
        *reinterpret_cast<u32x2_t *>(dst) = u32x2_t{v[0], v[1]};
        *reinterpret_cast<u32x2_t *>(dst + 4) = u32x2_t{v[2], v[3]};
    };

    // With 256 state columns the registers hold no tile in flight.
    constexpr bool kAhead = N <= 128 || !OUT;
    if (kAhead && tokens > 0)
        fetch(0);
    // lane parts of the LDS addresses: the transposing reads of b and x, the plain reads of c
    const uint32_t b_tr = lds_addr(&sh.b[4 * half + 8 * (l16 >> 2)][16 * odd + 4 * (l16 & 3)]);
    const int kappa = 4 * odd + (l16 & 3);
    const uint32_t x_tr = lds_addr(&sh.x[4 * half + 8 * (l16 >> 2)][wave * 32 + 16 * (kappa & 1) + 4 * (kappa >> 1)]);

    for (int tt = 0; tt < tokens; tt += TM) {
        if (!kAhead)
            fetch(tt);
#pragma unroll
        for (int k = 0; k < kLoadB; ++k) {
            if (bt0 < SB) {
                put(&sh.b[bt0 + k * SB][bc0], rb[k]);
                if constexpr (OUT)
                    put(&sh.c[bt0 + k * SB][bc0], rc[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kLoadX; ++k) {
            put(&sh.x[xt0 + k * SX][xc0], rx[k]);
        }
        int g;       // of token tt + lane within its chunk, in units of
        float unit;  // this many bits (the chunk's lanes share it)
        {
            const float raw = bf16_to_f32(static_cast<uint16_t>(rdt)) + dt_bias;
            const float dt = tt + lane < tokens ? (p.softplus ? softplus_f32(raw) : raw) : 0.0f;
            const float a = fmaxf(rate * dt, -160.0f);
            const float abs_sum = prefix32(fabsf(a));
            const float s0 = read_lane(abs_sum, 31), s1 = read_lane(abs_sum, 63);
            // 2^e <= sum < 2^(e + 1): a unit of 2^(e - 29)
            const uint32_t e = __float_as_uint(fmaxf(lane < 32 ? s0 : s1, 0x1p-60f)) & 0x7f800000u;
            unit = __uint_as_float(e - (29u << 23));
            g = prefix32(static_cast<int>(rintf(a * __uint_as_float((254u << 23) - e + (29u << 23)))));
            sh.g[wave][lane] = g;
            sh.d[wave][lane] = dt;
            sh.w[wave][lane] = dt * exp2_f32(after32(a, lane));
        }
        lds_barrier();
        if (kAhead && tt + TM < tokens)
            fetch(tt + TM);
        if constexpr (OUT) {
            // c b^T: wave w forms rows 16 (w >> 1 & 1) .. of t, columns 16 (w & 1) .. of s of chunk w >> 2
            const int q = wave >> 2, ts = 16 * ((wave >> 1) & 1), ss = 16 * (wave & 1);
            if (ss > ts) {
                *reinterpret_cast<f32x4_t *>(&sh.cb[q][ts + l16][ss + 4 * (lane >> 4)]) = f32x4_t{0, 0, 0, 0};
            } else {
                f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    const uint16_t *pb = &sh.b[CH * q + ss + l16][32 * k + 8 * (lane >> 4)];
                    const uint16_t *pc = &sh.c[CH * q + ts + l16][32 * k + 8 * (lane >> 4)];
                    const bf16x8_t vb = cat8(*reinterpret_cast<const u32x2_t *>(pb), *reinterpret_cast<const u32x2_t *>(pb + 4));
                    const bf16x8_t vc = cat8(*reinterpret_cast<const u32x2_t *>(pc), *reinterpret_cast<const u32x2_t *>(pc + 4));
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, vc, acc, 0, 0, 0);
                }
                // lane holds t = ts + l16, s = ss + 4 (lane / 16) + r; the tokens
                // after t are 0 here (ss < ts leaves none)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = ss == ts && 4 * (lane >> 4) + r > l16 ? 0.0f : acc[r];
                *reinterpret_cast<f32x4_t *>(&sh.cb[q][ts + l16][ss + 4 * (lane >> 4)]) = acc;
            }
            lds_barrier();
        }
#pragma unroll 1
        for (int q = 0; q < TM / CH; ++q) {
            const int r0 = CH * q;
            if (tt + r0 >= tokens || !active)
                break;
            const float bits = read_lane(unit, r0);
            const float total = bits * static_cast<float>(__builtin_amdgcn_readlane(g, r0 + CH - 1));
            bf16x8_t xa[2];  // x_s, column l32, tokens in contraction order
#pragma unroll
            for (int j = 0; j < 2; ++j)
                xa[j] = cat8(lds_tr(x_tr + 2 * kXPitch * (r0 + 2 * j)), lds_tr(x_tr + 2 * kXPitch * (r0 + 2 * j + 1)));

            if constexpr (OUT) {
                f32x16_t y;
#pragma unroll
                for (int r = 0; r < 16; ++r) y[r] = 0.0f;
                // S c_t
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint16_t *pc = &sh.c[r0 + l32][32 * nt + 16 * j + 4 * half];
                        const bf16x8_t vc = cat8(*reinterpret_cast<const u32x2_t *>(pc), *reinterpret_cast<const u32x2_t *>(pc + 8));
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = s[nt][8 * j + e];
                        bf16x8_t hi, lo;
                        split8(v, &hi, &lo);
                        y = mfma(hi, vc, y);
                        y = mfma(lo, vc, y);
                    }
                const int gt = sh.g[wave][r0 + l32];
                const float eg = exp2_f32(bits * static_cast<float>(gt));
#pragma unroll
                for (int r = 0; r < 16; ++r) y[r] *= eg;
                // M[t, s], t = l32, s = 8 i + 4 half + e; c b^T is 0 for s > t,
                // where the factor only has to stay finite
                float m[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s0 = 8 * i + 4 * half;
                    const f32x4_t cb = *reinterpret_cast<const f32x4_t *>(&sh.cb[q][l32][s0]);
                    const i32x4_t gs = *reinterpret_cast<const i32x4_t *>(&sh.g[wave][r0 + s0]);
                    const f32x4_t ds = *reinterpret_cast<const f32x4_t *>(&sh.d[wave][r0 + s0]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float span = fminf(bits * static_cast<float>(gt - gs[e]), 120.0f);
                        m[i][e] = fmaf(cb[e] * ds[e], exp2_f32(span), diag[4 * i + e]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = m[e & 3][2 * j + (e >> 2)];
                    bf16x8_t hi, lo;
                    split8(v, &hi, &lo);
                    y = mfma(xa[j], hi, y);
                    y = mfma(xa[j], lo, y);
                }
                if (tt + r0 + l32 < tokens) {
                    float f[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) f[r] = y[r];
                    if (zp) {
                        float z[16];
                        unpack8(*reinterpret_cast<const u32x4_a2 *>(zp), z);
                        unpack8(*reinterpret_cast<const u32x4_a2 *>(zp + 8), z + 8);
#pragma unroll
                        for (int r = 0; r < 16; ++r) f[r] *= silu_f32(z[r]);
                    }
                    *reinterpret_cast<u32x4_t *>(op) = pack8(f);
                    *reinterpret_cast<u32x4_t *>(op + 8) = pack8(f + 8);
                }
                if (zp)
                    zp += CH * p.zt;
                op += CH * p.H * p.P;
            }

            // S <- 2^total S + (w x) b^T
            bf16x8_t whi[2], wlo[2];
            {
                float w[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4_t v = *reinterpret_cast<const f32x4_t *>(&sh.w[wave][r0 + 8 * i + 4 * half]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[i][e] = v[e];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[8];
                    unpack8(__builtin_bit_cast(u32x4_t, xa[j]), v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= w[e & 3][2 * j + (e >> 2)];
                    split8(v, &whi[j], &wlo[j]);
                }
            }
            const float keep = exp2_f32(total);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[nt][r] *= keep;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t a = b_tr + 2 * kPitch * (r0 + 2 * j) + 64 * nt;
                    const bf16x8_t vb = cat8(lds_tr(a), lds_tr(a + 2 * kPitch));
                    s[nt] = mfma(vb, whi[j], s[nt]);
                    s[nt] = mfma(vb, wlo[j], s[nt]);
                }
            }
            log_sum += total;
        }
        lds_barrier();
    }

    if (!active)
        return;
    if constexpr (OUT) {
        if (last && p.final_state)
            store_state<N>(p.final_state, p.final_kind, state_at, s);
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4_t *>(slab + (4 * nt + i) * 256) =
                    f32x4_t{s[nt][4 * i], s[nt][4 * i + 1], s[nt][4 * i + 2], s[nt][4 * i + 3]};
        if (colblk == 0 && lane == 0)
            p.logs[slot * p.H + h] = log_sum;
    }
}

// The states in front of the segments, in order: start_0 = the initial state,
// start_(k+1) = 2^(log decay of k) start_k + own state of k, each over its
// segment's slab.  A thread carries four elements of one (sequence, head).
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void ssm_join_kernel(SsmParams p, int64_t quads)
{
    const int64_t per = (quads + kJoinThreads - 1) / kJoinThreads;
    const int64_t chain = blockIdx.x / per;
    const int64_t q = (blockIdx.x - chain * per) * kJoinThreads + threadIdx.x;  // quad within the head's slab
    const int64_t n = chain / p.H, h = chain - n * p.H;
    int64_t slot, len;
    if (p.seqs.cu) {
        const int64_t a = clamp_offset(p.seqs, n), b = clamp_offset(p.seqs, n + 1);
        slot = a / p.seg + n;
        len = b > a ? b - a : 0;
    } else {
        slot = n * (p.seqs.T > 0 ? (p.seqs.T + p.seg - 1) / p.seg : 1);
        len = p.seqs.T;
    }
    const int64_t count = len > 0 ? (len + p.seg - 1) / p.seg : 1;
    if (q >= quads)
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
    float *slab = p.slabs + (slot * p.H + h) * p.P * p.N + 4 * q;
    const float *logs = p.logs + slot * p.H + h;
    for (int64_t k = 0; k + 1 < count; ++k) {
        const f32x4_t own = *reinterpret_cast<const f32x4_t *>(slab + k * step);
        const float keep = exp2_f32(logs[k * p.H]);
        *reinterpret_cast<f32x4_t *>(slab + k * step) = run;
#pragma unroll
        for (int e = 0; e < 4; ++e) run[e] = fmaf(keep, run[e], own[e]);
    }
    *reinterpret_cast<f32x4_t *>(slab + (count - 1) * step) = run;
}

template <int N>
hipError_t launch(const SsmParams &p, hipStream_t stream)
{
    const int units = static_cast<int>(p.H / p.G * (p.P / 32)), ublocks = (units + NW - 1) / NW;
    const int64_t blocks = tile_slots(p.seqs, p.seg) * p.G * ublocks;
    const int64_t quads = p.P * N / 4, join = p.seqs.N * p.H * ((quads + kJoinThreads - 1) / kJoinThreads);
    if (blocks > INT32_MAX || join > INT32_MAX)
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
