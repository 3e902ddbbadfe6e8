// The gated delta rule with one decay per head in tiles of 64 tokens, on matrix
// instructions.  Per head, with G_t the sum of the log decays of a tile up to
// and with token t, S the state [K, V] in front of it, and for its tokens
//   A[t,s] = beta_t 2^(G_t - G_s) k_t . k_s  (s < t),  P[t,s] = 2^(G_t - G_s) q_t . k_s  (s <= t),
//   (I + A) U = beta (V - 2^G K S)
//   out = scale (2^G Q S + P U)
//   S <- 2^(G_63) S + sum_s 2^(G_63 - G_s) k_s u_s^T
// No exponent is positive, so nothing overflows however strong the decay.  (I +
// A) is solved in blocks of 16 tokens: block by block what earlier ones give is
// taken off, and what is left multiplied by the inverse of the diagonal block,
// which forward substitution gives.
//
// A workgroup of eight waves owns a (sequence, head) and up to 128 of its V
// columns, 16 a wave, with the fp32 state [K, 16] in accumulators from the
// sequence's first token to its last.  K, Q, V, A and P of a tile are in LDS,
// shared by the waves: wave 0 forms and inverts the diagonal blocks of A, the
// others the remaining blocks of A and P, and then each wave goes through the
// tile alone.  The next tile's rows are loaded meanwhile, its decays and
// strengths worked out by the last wave.
//
// Operands.  In v_mfma_f32_16x16x32_bf16 lane (r = lane % 16, g = lane / 16)
// holds row / column r, slots 8 g .. 8 g + 7, and accumulator register i is row
// 4 g + i of column r.  Which contraction index a slot stands for is free as
// long as both operands agree, so with slot 8 g + 4 a + i standing for index 16 a
// + 4 g + i two accumulators on top of each other are an operand as they stand:
// S over k, U over tokens, as right factor and, transposed, as left.  K, Q and P
// lie in LDS in that order, 32 at a time, so that a lane's slots are adjacent.
// out comes transposed, four adjacent columns of a token to a lane.  In
// v_mfma_f32_16x16x4_f32 of the solve, step i takes row 4 g + i: accumulator
// register i again.
//
// Numerics.  k, q and v are bf16 and enter as they are.  Of what is fp32, S
// enters K S and the weighted U enters S as three bf16 parts, which hold all 24
// bits; the solve is fp32 throughout.  S enters Q S, and P and U enter P U, as two
// parts, good to 2^-17 (out is rounded to 2^-8); of their products the last times
// the last is left out.  G is summed in 64 bits and kept as two floats, since
// differences of sums lose a small decay beside a strong one.
//
// What is not finite (or beyond 2^120, where parts overflow) must not reach
// earlier tokens through the zeros of a block's upper half: such elements of U
// and all behind them in their column are taken for 0, and the column's outputs
// from there on, and its state, are made NaN.
#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int TM = 64, NB = TM / 16;  // tokens and blocks of a tile
constexpr int kWaves = 8, kThreads = 64 * kWaves, kColumns = 16 * kWaves;
constexpr float kLarge = 0x1p120f;
constexpr float kGone = -1000.0f;  // log decay below which nothing is left, also in 64 tokens' sum

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
__device__ __forceinline__ u32x4_t cat(u32x2_t a, u32x2_t b) { return u32x4_t{a[0], a[1], b[0], b[1]}; }
__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
// c + a b of 16 x 16 fp32 blocks: a's rows lie over the lanes (four adjacent
// elements each), b is an accumulator.
__device__ __forceinline__ f32x4_t mfma_f32(f32x4_t a, f32x4_t b, f32x4_t c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}
// Workgroup barrier that orders LDS only: loads to registers stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
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
// v as a sum of bf16 numbers, each what is left rounded to nearest: two leave
// 2^-17 of v at most, three hold its 24 bits.
template <int PARTS>
__device__ __forceinline__ void split(f32x4_t v, u32x2_t (&h)[PARTS])
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float a = v[2 * j], b = v[2 * j + 1];
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            h[k][j] = pack_bf16x2(a, b);
            a -= lo_f32(h[k][j]);
            b -= hi_f32(h[k][j]);
        }
    }
}
__device__ __forceinline__ uint32_t size_bits(f32x4_t v)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}
__device__ __forceinline__ bool odd(f32x4_t v) { return size_bits(v) > __float_as_uint(kLarge); }

// The sum over the wave's lanes up to and with each lane.
__device__ __forceinline__ double prefix(double x, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double y = __shfl_up(x, d);
        x += lane >= d ? y : 0.0;
    }
    return x;
}

// Rows of K and Q: 20 mod 64 dwords apart, which puts eight rows' 16 bytes in
// distinct banks, and nearly all of what a transposing read takes.
template <int K>
constexpr int kRowPitch = K == 64 ? 168 : K + 40;
constexpr int kVPitch = kColumns + 16, kAPitch = TM + 4, kPPitch = TM + 8;

template <int K>
struct Shared {
    alignas(16) uint16_t k[TM][kRowPitch<K>];
    alignas(16) uint16_t q[TM][kRowPitch<K>];
    alignas(16) uint16_t v[TM][kVPitch];
    alignas(16) float a[TM][kAPitch];         // -A below the diagonal blocks, the inverses on it
    alignas(16) uint16_t p[2][TM][kPPitch];   // two parts of P
    // for the tiles in turn: G in two floats, 2^G, 2^(G_63 - G), beta
    alignas(16) float g[2][2][TM], decay[2][TM], left[2][TM], beta[2][TM];
    float total[2];                           // 2^(G_63)
};

template <int K>
__global__ __launch_bounds__(kThreads) void delta_chunk_kernel(DeltaParams p, int vblocks, int columns)
{
    constexpr int KT = K / 16, KSTEP = K / 32, PK = K / 8;  // state tiles; steps over k; 16-byte pieces of a row
    constexpr int kLoad = TM * PK / kThreads;               // pieces of K (and of Q) a thread loads
    constexpr int kLoadV = TM * kColumns / 8 / kThreads;
    constexpr bool kAhead = K <= 128;  // with 256 state rows the registers hold no tile in flight
    static_assert(kLoad >= 1 && kLoadV >= 1, "whole rounds of loads");
    __shared__ __align__(16) Shared<K> sh;

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t chain = blockIdx.x / static_cast<uint32_t>(vblocks), vb = blockIdx.x - chain * static_cast<uint32_t>(vblocks);
    const int64_t n = chain / static_cast<uint32_t>(p.H), h = chain - static_cast<uint32_t>(n) * static_cast<uint32_t>(p.H);
    const int64_t grp = h / (p.H / p.G);
    int64_t row = n;
    int begin = 0, end = static_cast<int>(p.seqs.T);
    if (p.seqs.cu) {
        row = 0;
        begin = static_cast<int>(clamp_offset(p.seqs, n));
        end = static_cast<int>(clamp_offset(p.seqs, n + 1));
    }
    const int tokens = end > begin ? end - begin : 0;
    const int col0 = static_cast<int>(vb) * columns, width = static_cast<int>(p.V) - col0 < columns ? static_cast<int>(p.V) - col0 : columns;
    const bool active = 16 * wave < width;  // waves without columns help with what is shared
    const int col = col0 + 16 * wave;

    // the state: tile t's register i is k = 16 t + 4 g + i of column r
    f32x4_t s[KT];
    const int64_t slab = ((n * p.H + h) * p.V + col + r) * K + 4 * g;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        s[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (active) {
            if (p.init_kind == kFp32) {
                s[t] = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p.init_state) + slab + 16 * t);
            } else if (p.init_kind == kBf16) {
                const u32x2_t v = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(p.init_state) + slab + 16 * t);
                s[t] = f32x4_t{lo_f32(v[0]), hi_f32(v[0]), lo_f32(v[1]), hi_f32(v[1])};
            }
        }
    }

    const float rate = -expf(p.A_log[h]) * kLog2eF, bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    const char *kbase = reinterpret_cast<const char *>(p.k + row * p.kb + static_cast<int64_t>(begin) * p.kt + grp * K);
    const char *qbase = reinterpret_cast<const char *>(p.q + row * p.qb + static_cast<int64_t>(begin) * p.qt + grp * K);
    const char *vbase = reinterpret_cast<const char *>(p.v + row * p.vb + static_cast<int64_t>(begin) * p.vt + h * p.V + col0);
    const uint16_t *gbase = p.g + row * p.gb + static_cast<int64_t>(begin) * p.gt + h;
    const uint16_t *bbase = p.beta + row * p.bb + static_cast<int64_t>(begin) * p.bt + h;
    uint16_t *obase = p.out + ((row * p.seqs.T + begin) * p.H + h) * p.V + col;

    // A tile's rows on their way from memory to LDS; rows past the end are zeros.
    u32x4_t nk[kLoad], nq[kLoad], nv[kLoadV];
    const auto load = [&](int t0) {
        const int left = tokens - t0, me = here(tid);
        const char *kp = kbase + static_cast<int64_t>(t0) * p.kt * 2, *qp = qbase + static_cast<int64_t>(t0) * p.qt * 2;
        const char *vp = vbase + static_cast<int64_t>(t0) * p.vt * 2;
#pragma unroll
        for (int i = 0; i < kLoad; ++i) {
            const int piece = me + kThreads * i, t = piece / PK, c = piece % PK, in = t < left ? t : left - 1;
            const u32x4_t x = *reinterpret_cast<const u32x4_a2 *>(kp + static_cast<uint32_t>(in) * static_cast<uint32_t>(2 * p.kt) + 16 * c);
            const u32x4_t y = *reinterpret_cast<const u32x4_a2 *>(qp + static_cast<uint32_t>(in) * static_cast<uint32_t>(2 * p.qt) + 16 * c);
            nk[i] = t < left ? x : u32x4_t{0, 0, 0, 0};
            nq[i] = t < left ? y : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kLoadV; ++i) {
            const int piece = me + kThreads * i, t = piece / (kColumns / 8), c = piece % (kColumns / 8);
            const int in = t < left ? t : left - 1, at = 8 * c < width ? c : 0;
            const u32x4_t x = *reinterpret_cast<const u32x4_a2 *>(vp + static_cast<uint32_t>(in) * static_cast<uint32_t>(2 * p.vt) + 16 * at);
            nv[i] = t < left ? x : u32x4_t{0, 0, 0, 0};
        }
    };
    const auto store = [&] {
        const int me = here(tid);
#pragma unroll
        for (int i = 0; i < kLoad; ++i) {
            // channels 8 m .. 8 m + 7 of 32: two runs of four, in the order of the slots
            const int piece = me + kThreads * i, t = piece / PK, c = piece % PK;
            const int at = 32 * (c / 4) + 16 * (c % 2) + 4 * (c % 4 / 2);
            *reinterpret_cast<u32x2_t *>(&sh.k[t][at]) = u32x2_t{nk[i][0], nk[i][1]};
            *reinterpret_cast<u32x2_t *>(&sh.k[t][at + 8]) = u32x2_t{nk[i][2], nk[i][3]};
            *reinterpret_cast<u32x2_t *>(&sh.q[t][at]) = u32x2_t{nq[i][0], nq[i][1]};
            *reinterpret_cast<u32x2_t *>(&sh.q[t][at + 8]) = u32x2_t{nq[i][2], nq[i][3]};
        }
#pragma unroll
        for (int i = 0; i < kLoadV; ++i) {
            const int piece = me + kThreads * i, t = piece / (kColumns / 8), c = piece % (kColumns / 8);
            *reinterpret_cast<u32x4_t *>(&sh.v[t][8 * c]) = nv[i];
        }
    };
    // The decays and strengths of a tile, a token a lane.
    const auto gates = [&](int t0, int buf) {
        const int t = t0 + lane, in = t < tokens ? t : tokens - 1;
        const float raw = lo_f32(gbase[static_cast<int64_t>(in) * p.gt]) + bias;
        const float logit = lo_f32(bbase[static_cast<int64_t>(in) * p.bt]);
        float a = rate * softplus_f32(raw, dt_plain_above(1));
        a = a < kGone ? kGone : a;
        const double sum = prefix(t < tokens ? static_cast<double>(a) : 0.0, lane);
        const float hi = static_cast<float>(sum), lo = static_cast<float>(sum - static_cast<double>(hi));
        const float last_hi = __shfl(hi, 63), last_lo = __shfl(lo, 63);
        sh.g[buf][0][lane] = hi;
        sh.g[buf][1][lane] = lo;
        sh.decay[buf][lane] = exp2_f32(hi + lo);
        sh.left[buf][lane] = exp2_f32((last_hi - hi) + (last_lo - lo));
        sh.beta[buf][lane] = t < tokens ? sigmoid_f32(logit) : 0.0f;
        if (lane == 63)
            sh.total[buf] = exp2_f32(hi + lo);
    };
    // Blocks (b, c) of A and P: lane r is token 16 b + r, its registers tokens 16 c + 4 g + i before it.
    const auto block_products = [&](int b, int c, int buf, bool with_a, bool with_p) {
        f32x4_t kk = {0.0f, 0.0f, 0.0f, 0.0f}, qk = kk;
#pragma unroll
        for (int e = 0; e < KSTEP; ++e) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t *>(&sh.k[16 * c + r][32 * e + 8 * g]);
            if (with_a)
                kk = mfma(x, *reinterpret_cast<const u32x4_t *>(&sh.k[16 * b + r][32 * e + 8 * g]), kk);
            if (with_p)
                qk = mfma(x, *reinterpret_cast<const u32x4_t *>(&sh.q[16 * b + r][32 * e + 8 * g]), qk);
        }
        const int i = 16 * b + r, j = 16 * c + 4 * g;
        const float hi = sh.g[buf][0][i], lo = sh.g[buf][1][i];
        const f32x4_t hj = *reinterpret_cast<const f32x4_t *>(&sh.g[buf][0][j]), lj = *reinterpret_cast<const f32x4_t *>(&sh.g[buf][1][j]);
        f32x4_t x, y;
        const float strength = with_a ? -sh.beta[buf][i] : 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float f = exp2_f32((hi - hj[m]) + (lo - lj[m]));
            x[m] = j + m < i ? strength * f * kk[m] : 0.0f;
            y[m] = j + m <= i ? f * qk[m] : 0.0f;
        }
        if (with_a)
            *reinterpret_cast<f32x4_t *>(&sh.a[i][j]) = x;
        if (with_p) {
            u32x2_t parts[2];
            split<2>(y, parts);
            const int at = 32 * (c / 2) + 8 * g + 4 * (c % 2);
            *reinterpret_cast<u32x2_t *>(&sh.p[0][i][at]) = parts[0];
            *reinterpret_cast<u32x2_t *>(&sh.p[1][i][at]) = parts[1];
        }
    };
    // The inverses of the diagonal blocks I + A by forward substitution: lane (g, r)
    // has column r of block g, X_i = e_i - sum_(m < i) A_im X_m.
    const auto invert = [&] {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = i == here(r) ? 1.0f : 0.0f;
#pragma unroll
            for (int m4 = 0; m4 < i; m4 += 4) {
                const f32x4_t a = *reinterpret_cast<const f32x4_t *>(&sh.a[16 * g + i][16 * g + m4]);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (m4 + m < i)
                        x[i] = fmaf(a[m], x[m4 + m], x[i]);  // -A is stored
            }
            if (i % 4 == 3)  // no more rows of A in registers at once
                asm volatile("" : "+v"(x[i]), "+v"(x[i - 1]), "+v"(x[i - 2]), "+v"(x[i - 3])::"memory");
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) sh.a[16 * g + i][16 * g + r] = x[i];
    };

    // what P U reads of blocks above the diagonal
    for (int i = tid; i < 2 * TM * kPPitch / 2; i += kThreads) reinterpret_cast<uint32_t *>(sh.p)[i] = 0;
    if (tokens > 0) {
        load(0);
        if (wave == kWaves - 1)
            gates(0, 0);
        store();
    }
    int buf = 0;
    for (int t0 = 0; t0 < tokens; t0 += TM, buf ^= 1) {
        lds_barrier();
        const bool more = t0 + TM < tokens;
        if (kAhead && more)
            load(t0 + TM);
        if (wave == 0) {
#pragma unroll 1
            for (int b = 0; b < NB; ++b) block_products(b, b, buf, true, false);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            invert();
        } else {
            // 6 blocks below the diagonal, of A and P, and 4 on it, of P
#pragma unroll 1
            for (int i = wave - 1; i < 10; i += kWaves - 1) {
                const int b = i < 6 ? (i < 1 ? 1 : i < 3 ? 2 : 3) : i - 6, c = i < 6 ? i - (b == 1 ? 0 : b == 2 ? 1 : 3) : i - 6;
                block_products(b, c, buf, i < 6, true);
            }
            if (wave == kWaves - 1 && more)
                gates(t0 + TM, buf ^ 1);
        }

        // K S and Q S: rows are tokens of K S, columns of (Q S)^T
        f32x4_t u[NB], o[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) u[b] = o[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (active) {
#pragma unroll
            for (int e = 0; e < KSTEP; ++e) {
                u32x2_t x[3], y[3];
                split<3>(s[2 * e], x);
                split<3>(s[2 * e + 1], y);
                const u32x4_t s0 = cat(x[0], y[0]), s1 = cat(x[1], y[1]), s2 = cat(x[2], y[2]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const u32x4_t kr = *reinterpret_cast<const u32x4_t *>(&sh.k[16 * b + r][32 * e + 8 * g]);
                    const u32x4_t qr = *reinterpret_cast<const u32x4_t *>(&sh.q[16 * b + r][32 * e + 8 * g]);
                    u[b] = mfma(kr, s0, u[b]);
                    o[b] = mfma(s0, qr, o[b]);
                    u[b] = mfma(kr, s1, u[b]);
                    o[b] = mfma(s1, qr, o[b]);
                    u[b] = mfma(kr, s2, u[b]);
                }
                fence();
            }
        }
        lds_barrier();
        if (active) {
            const uint32_t vaddr = lds_addr(&sh.v[4 * g + r / 4][16 * wave + 4 * (r & 3)]);
            int poison = TM;  // of column r: the first token whose U is not finite
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const u32x2_t vr = lds_tr(vaddr + 32 * b * kVPitch);
                const f32x4_t d = *reinterpret_cast<const f32x4_t *>(&sh.decay[buf][16 * b + 4 * g]);
                const f32x4_t beta = *reinterpret_cast<const f32x4_t *>(&sh.beta[buf][16 * b + 4 * g]);
                const f32x4_t v = {lo_f32(vr[0]), hi_f32(vr[0]), lo_f32(vr[1]), hi_f32(vr[1])};
#pragma unroll
                for (int i = 0; i < 4; ++i) u[b][i] = beta[i] * fmaf(-d[i], u[b][i], v[i]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // takes out what is odd in the block (16 tokens of each column), from its first on
                const auto scrub = [&](f32x4_t &x) {
                    if (!__any(odd(x) || poison < TM))
                        return;
                    int first = poison;
#pragma unroll
                    for (int i = 3; i >= 0; --i)
                        if ((__float_as_uint(x[i]) & 0x7fffffffu) > __float_as_uint(kLarge) && 16 * b + 4 * g + i < first)
                            first = 16 * b + 4 * g + i;
                    const int other = __shfl_xor(first, 16), both = other < first ? other : first;
                    const int far = __shfl_xor(both, 32);
                    poison = far < both ? far : both;
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = 16 * b + 4 * g + i >= poison ? 0.0f : x[i];
                };
                f32x4_t rest = u[b];
#pragma unroll
                for (int c = 0; c < b; ++c)
                    rest = mfma_f32(*reinterpret_cast<const f32x4_t *>(&sh.a[16 * b + r][16 * c + 4 * g]), u[c], rest);
                scrub(rest);
                u[b] = mfma_f32(*reinterpret_cast<const f32x4_t *>(&sh.a[16 * b + r][16 * b + 4 * g]), rest, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
                scrub(u[b]);
            }

            fence();
            // out
            u32x2_t up[NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) split<2>(u[b], up[b]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                o[b] *= sh.decay[buf][16 * b + r];
#pragma unroll
                for (int e = 0; e <= b / 2; ++e) {
                    const u32x2_t none = {0, 0};
                    const bool two = 2 * e + 1 <= b;
                    const u32x4_t u0 = cat(up[2 * e][0], two ? up[2 * e + 1][0] : none), u1 = cat(up[2 * e][1], two ? up[2 * e + 1][1] : none);
                    const u32x4_t p0 = *reinterpret_cast<const u32x4_t *>(&sh.p[0][16 * b + r][32 * e + 8 * g]);
                    const u32x4_t p1 = *reinterpret_cast<const u32x4_t *>(&sh.p[1][16 * b + r][32 * e + 8 * g]);
                    o[b] = mfma(u0, p0, o[b]);
                    o[b] = mfma(u1, p0, o[b]);
                    o[b] = mfma(u0, p1, o[b]);
                }
                o[b] *= p.scale;
            }
            const bool poisoned = __any(poison < TM);
            if (poisoned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = __shfl(poison, 4 * g + i);
#pragma unroll
                    for (int b = 0; b < NB; ++b) o[b][i] = 16 * b + r >= from ? __builtin_nanf("") : o[b][i];
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (t0 + 16 * b + r < tokens)
                    *reinterpret_cast<u32x2_t *>(obase + static_cast<int64_t>(t0 + 16 * b + r) * p.H * p.V + 4 * g) =
                        u32x2_t{pack_bf16x2(o[b][0], o[b][1]), pack_bf16x2(o[b][2], o[b][3])};

            fence();
            // the state
            u32x2_t w[NB][3];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const f32x4_t left = *reinterpret_cast<const f32x4_t *>(&sh.left[buf][16 * b + 4 * g]);
                split<3>(u[b] * left, w[b]);
            }
            const float total = sh.total[buf];
            const uint32_t kaddr = lds_addr(&sh.k[4 * g + r / 4][8 * (r & 3)]);
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                s[t] *= total;
#pragma unroll
                for (int e = 0; e < NB / 2; ++e) {
                    const uint32_t at = kaddr + 2 * (32 * (t / 2) + 4 * (t % 2)) + 2 * 32 * e * kRowPitch<K>;
                    const u32x4_t kr = cat(lds_tr(at), lds_tr(at + 2 * 16 * kRowPitch<K>));
#pragma unroll
                    for (int k = 0; k < 3; ++k) s[t] = mfma(kr, cat(w[2 * e][k], w[2 * e + 1][k]), s[t]);
                }
                if (t % 2 == 1)
                    fence();
            }
            if (poisoned) {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] = poison < TM ? __builtin_nanf("") : s[t][i];
            }
        }
        if (more) {
            if (!kAhead)
                load(t0 + TM);
            lds_barrier();
            store();
        }
    }

    if (!p.final_state || !active)
        return;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        if (p.final_kind == kFp32)
            *reinterpret_cast<f32x4_t *>(static_cast<float *>(p.final_state) + slab + 16 * t) = s[t];
        else
            *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(p.final_state) + slab + 16 * t) =
                u32x2_t{pack_bf16x2(s[t][0], s[t][1]), pack_bf16x2(s[t][2], s[t][3])};
    }
}

template <int K>
hipError_t launch(const DeltaParams &p, hipStream_t stream)
{
    const int columns = static_cast<int>(p.V < kColumns ? p.V : kColumns);
    const int64_t vblocks = (p.V + columns - 1) / columns, blocks = p.seqs.N * p.H * vblocks;
    if (!grid_fits(blocks, kThreads))
        return hipErrorInvalidConfiguration;
    delta_chunk_kernel<K><<<dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream>>>(p, static_cast<int>(vblocks), columns);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunk(const DeltaParams &p, hipStream_t stream)
{
    switch (p.K) {
    case 64: return launch<64>(p, stream);
    case 128: return launch<128>(p, stream);
    case 256: return launch<256>(p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace layer
}  // namespace kda
