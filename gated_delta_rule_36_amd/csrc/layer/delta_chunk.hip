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
// A workgroup of twelve waves owns a (sequence, head) and up to 128 of its V
// columns.  Eight carry 16 columns of the fp32 state [K, 16] each, in accumulators
// from the sequence's first token to its last; four prepare the tiles, which lie
// in LDS twice over.  Two barriers a tile:
// - state waves: K S and Q S of the tile, V's own columns through LDS.  Preparing
//   waves: the inverses of the diagonal blocks of A (one wave), the next tile's
//   rows from registers to LDS with its decays and strengths (another one), the
//   loads of the one after.
// - state waves: what is left of beta (V - 2^G K S), U, out, the state.  Preparing
//   waves: the next tile's blocks of A and P.
// Preparation takes no state, so all of it leaves the chain of tiles that has to
// be gone through in order: 8 x 16384 tokens took 2.22 ms with the state waves doing it all, 1.81 after.
//
// Few long chains are cut into segments, for which the rule is an affine map of
// the state: a pass forms every segment's own end and what it makes of each unit
// vector, K columns more; a second kernel joins them in fp32; the output pass
// starts each segment from what that gives.  8191 tokens of 12 heads of 64 x 96:
// 391 us whole, 107 in 10 segments, of which the join is 8 and either pass half the rest.
//
// What bounds it: 8 x 16384 tokens of 32 heads of 128 x 128 take 1.69 to 1.74 ms (1.9 TB/s, 38 % of
// a large copy's rate), 14000 cycles a tile, of which a SIMD's matrix
// instructions are busy 7550, vector ones 4900 and LDS 5400, beside each other only
// where a second wave is there; and a chip this busy runs at 1.9 instead of 2.4 GHz.
// Tried and lost: 32 columns a state wave (1795 us against 1700), more priority for
// the preparing waves (1757 against 1725), one of a SIMD's two state waves half a
// tile ahead of the other (1768 against 1730: the second half of a tile takes two
// thirds of it), the inverses in the same half as the blocks (packed 365 against 350),
// the solve's products below the diagonal by bf16 parts (1773 against 1755, packed 356
// against 350: a third fewer matrix cycles there, but the parts stand in the chain), the
// output's products of all blocks in turn (packed 355 against 345).
//
// Operands.  In v_mfma_f32_16x16x32_bf16 lane (r = lane % 16, g = lane / 16)
// holds row / column r, slots 8 g .. 8 g + 7, and accumulator register i is row
// 4 g + i of column r.  Which contraction index a slot stands for is free as
// long as both operands agree, so two accumulators on top of each other are an
// operand as they stand, as right factor and, transposed, as left: S over k, with
// row 4 g + i of tile 2 e + a standing for k = 32 e + 8 g + 4 a + i, so that K and Q
// lie in LDS as in memory; and U over tokens, with slot 8 g + 4 a + i standing for
// token 16 a + 4 g + i of 32, the order in which P lies in LDS.  out comes
// transposed, four adjacent columns of a token to a lane.  In
// v_mfma_f32_16x16x4_f32 of the solve, step i takes row 4 g + i: accumulator
// register i again.
//
// Rows in LDS are 8 mod 16 dwords apart: 16 lanes' 16-byte pieces of 16 rows, four
// times, then take 6 cycles (10 at 4 mod 16, 34 at 0), and what a transposing read
// takes of K 6 (10 and 6).
//
// Numerics.  k, q and v are bf16 and enter as they are.  Of what is fp32, S
// enters K S and the weighted U enters S as three bf16 parts, which hold all 24
// bits; the solve is fp32 throughout.  S enters Q S, and P and U enter P U, as two
// parts, good to 2^-17 (out is rounded to 2^-8; bf16 outputs are 1.2e-4 of their norm
// off the rounded definition, 1.7e-3 off the definition either way); of their products
// the last times the last is left out.  Third parts of S and of U there and the product
// left out would take 1880 us for 1735 and leave 8.9e-5; of P they do not fit in LDS.
// One part of everything, the solve in fp32 as it is, takes 1227 us for 1690, packed 294
// for 340, long 94 for 107, at the price of the state's digits.  G is summed in 64 bits
// and kept as two floats, since differences of sums lose a small decay beside a strong one.
//
// What is not finite must not reach earlier tokens through the zeros of a
// block's upper half: where what U is solved from is not, it and all behind it in
// its column are taken for 0, and the column's outputs from there on, and its
// state, are made NaN.  So is U where it is not finite after all (a solve that
// overflows by itself: then also tokens of the same 16 before).
#include <cstddef>

#include "layer_device.h"

namespace kda {
namespace layer {
namespace {

// Waves with 16 columns of the state each, and waves that prepare tiles.
constexpr int kStateWaves = 8, kProducers = 4, kThreads = 64 * (kStateWaves + kProducers), kColumns = 16 * kStateWaves;
// Magnitudes from here on round to infinity as bf16 (or are not finite).
constexpr uint32_t kOddBits = 0x7f7f8000u;
constexpr float kGone = -1000.0f;  // log decay below which nothing is left, also in 64 tokens' sum

template <class T>
__device__ __forceinline__ T lds_load(uint32_t a)
{
    return *(const __attribute__((address_space(3))) T *)(uintptr_t)a;
}
__device__ __forceinline__ u32x4_t cat(u32x2_t a, u32x2_t b) { return u32x4_t{a[0], a[1], b[0], b[1]}; }
// The product over 16 slots, 4 g .. 4 g + 3 in a lane.
__device__ __forceinline__ f32x4_t mfma16(u32x2_t a, u32x2_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4_t, a), __builtin_bit_cast(s16x4_t, b), c, 0, 0, 0);
}
// c + a b of 16 x 16 fp32 blocks: a's rows lie over the lanes (four adjacent
// elements each), b is an accumulator.
__device__ __forceinline__ f32x4_t mfma_f32(f32x4_t a, f32x4_t b, f32x4_t c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
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
// 2^-17 of v at most, three hold its 24 bits.  What is left of both numbers of a
// pair comes from its rounded ones by a dot product with (-1, 0) or (0, -1), exact
// here, which takes the place of taking the pair apart and subtracting.  (A part
// that is not finite makes its neighbour's rest so, too.)
__device__ __forceinline__ float rest_of(uint32_t h, uint32_t which, float v)
{
    asm("" : "+s"(which));  // from a register: as an inline constant -1 does not stand for the pair (-1, 0)
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, h), __builtin_bit_cast(bf16x2_t, which), v, false);
}
template <int PARTS>
__device__ __forceinline__ void split(f32x4_t v, u32x2_t (&h)[PARTS])
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float a = v[2 * j], b = v[2 * j + 1];
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            h[k][j] = pack_bf16x2(a, b);
            if (k + 1 < PARTS) {
                a = rest_of(h[k][j], 0x0000bf80u, a);
                b = rest_of(h[k][j], 0xbf800000u, b);
            }
        }
    }
}
// The larger of two pairs of bf16 without their signs, each by itself.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_bf16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b & 0x7fff7fffu)));
}

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

// Lower blocks (b, c), c <= b, one after the other; of P two of them, side by side
// in the order of the slots (of an odd one out the second half is not used).
__device__ __forceinline__ constexpr int a_block(int b, int c) { return b * (b + 1) / 2 + c; }
__device__ __forceinline__ constexpr int p_block(int b, int e) { return (b / 2) * (b / 2 + 1) + (b % 2) * (b / 2 + 1) + e; }

template <int K, int TM>
struct LdsTile {
    static constexpr int NB = TM / 16, kPitch = K + 16, kAPitch = 24, kPPitch = 48;
    alignas(16) uint16_t k[TM][kPitch];
    alignas(16) uint16_t q[TM][kPitch];
    alignas(16) float a[a_block(NB - 1, NB - 1) + 1][16][kAPitch];               // -A below the diagonal, the inverses on it
    alignas(16) uint16_t p[2][p_block(NB - 1, (NB - 1) / 2) + 1][16][kPPitch];  // two parts of P
    // G in two floats, 2^G, 2^(G_last - G), beta; 2^G_last
    alignas(16) float g[2][TM], decay[TM], left[TM], beta[TM];
    float total;
};

template <int K, int TM>
struct Shared {
    LdsTile<K, TM> tile[2];
    alignas(16) uint16_t v[kStateWaves][TM][16];
};

// Where a workgroup's chain lies: a (sequence, head), or a segment of one.
struct Chain {
    int64_t n, h, grp, row;
    int begin, tokens, col0, width;  // its tokens, its columns
    int index;                       // of the segment
    bool several, last;              // one of several; the sequence's last
    int64_t slab;                    // the sequence's first slab
    bool valid;
};
// Rows of a slab: the state [V, K] at the end of the segment before, and behind it
// [K, K] what that segment makes of each unit vector.
__device__ __forceinline__ int64_t slab_row(const DeltaParams &p, int64_t slab, int64_t h, int64_t row)
{
    return ((slab * p.H + h) * (p.V + p.K) + row) * p.K;
}
__device__ __forceinline__ Chain find_chain(const DeltaParams &p, int all, int vblocks, int columns)
{
    Chain c;
    const uint32_t chain = blockIdx.x / static_cast<uint32_t>(vblocks), vb = blockIdx.x - chain * static_cast<uint32_t>(vblocks);
    const uint32_t slot = chain / static_cast<uint32_t>(p.H);
    c.h = chain - slot * static_cast<uint32_t>(p.H);
    c.grp = c.h / (p.H / p.G);
    c.col0 = static_cast<int>(vb) * columns;
    c.width = all - c.col0 < columns ? all - c.col0 : columns;
    if (p.seg == 0) {
        c.n = slot;
        if (p.seqs.cu && p.seqs.N <= kLaneSequences) {
            // the longest sequences first, so that the last workgroups to end are short ones: the lane whose
            // sequence as many others come before as the slot says
            const uint32_t lane = __lane_id();
            const LaneSequence q = lane_sequence(p.seqs, 1, lane);
            const int length = lane < p.seqs.N ? static_cast<int>(q.end - q.begin) : -1;
            int rank = 0;
            for (int m = 0; m < static_cast<int>(p.seqs.N); ++m) {
                const int other = __builtin_amdgcn_readlane(length, m);
                rank += other > length || (other == length && m < static_cast<int>(lane));
            }
            const uint64_t found = __ballot(lane < p.seqs.N && rank == static_cast<int>(slot));
            c.n = found ? __builtin_ctzll(found) : 0;
        }
        c.row = p.seqs.cu ? 0 : c.n;
        c.begin = p.seqs.cu ? static_cast<int>(clamp_offset(p.seqs, c.n)) : 0;
        const int end = p.seqs.cu ? static_cast<int>(clamp_offset(p.seqs, c.n + 1)) : static_cast<int>(p.seqs.T);
        c.tokens = end > c.begin ? end - c.begin : 0;
        c.index = 0;
        c.several = false;
        c.last = c.valid = true;
        c.slab = 0;
        return c;
    }
    const uint32_t seg = static_cast<uint32_t>(p.seg);
    const layer::Tile t = find_tile(p.seqs, seg, slot);
    const uint32_t t0 = t.index * seg, left = t.end - t.begin - t0;
    c.n = t.n;
    c.row = t.row;
    c.begin = static_cast<int>(t.begin + t0);
    c.last = left <= seg;
    c.tokens = static_cast<int>(c.last ? left : seg);
    c.index = static_cast<int>(t.index);
    c.several = t.end - t.begin > seg;
    c.slab = p.map.mul * (t.begin / seg) + p.map.add * t.n;
    c.valid = t.valid;
    return c;
}

// The waves that prepare tiles: rows of K and Q into LDS, decays and strengths,
// the blocks of A and P, the inverses of A's diagonal blocks.
template <int K, int TM, bool OUT>
struct Producer {
    static constexpr int NB = TM / 16, PK = K / 8;                 // 16-byte pieces of a row
    static constexpr int kRows = 64 * kProducers / PK, kLoad = TM / kRows;  // rows loaded at once, and how often
    static_assert(kLoad >= 1 && kLoad * kRows == TM, "whole rounds of loads");
    const DeltaParams &p;
    const Chain &ch;
    const int tid, lane, r, g, wave;
    float rate, bias;
    const char *kbase, *qbase;
    const uint16_t *gbase, *bbase;
    uint32_t koff, qoff;  // of a thread's piece of the first rows
    u32x4_t nk[kLoad], nq[kLoad];
    uint32_t ng, nb;

    __device__ __forceinline__ Producer(const DeltaParams &params, const Chain &chain, int t, int w)
        : p(params), ch(chain), tid(t), lane(t & 63), r(t & 15), g((t & 63) >> 4), wave(w)
    {
        rate = -expf(p.A_log[ch.h]) * kLog2eF;
        bias = p.dt_bias ? p.dt_bias[ch.h] : 0.0f;
        kbase = reinterpret_cast<const char *>(p.k + ch.row * p.kb + static_cast<int64_t>(ch.begin) * p.kt + ch.grp * K);
        qbase = reinterpret_cast<const char *>(p.q + ch.row * p.qb + static_cast<int64_t>(ch.begin) * p.qt + ch.grp * K);
        gbase = p.g + ch.row * p.gb + static_cast<int64_t>(ch.begin) * p.gt + ch.h;
        bbase = p.beta + ch.row * p.bb + static_cast<int64_t>(ch.begin) * p.bt + ch.h;
        koff = static_cast<uint32_t>(tid / PK) * static_cast<uint32_t>(2 * p.kt) + 16 * (tid % PK);
        qoff = static_cast<uint32_t>(tid / PK) * static_cast<uint32_t>(2 * p.qt) + 16 * (tid % PK);
    }

    // The tile's rows into registers; rows past the end are the last one, once more.
    __device__ __forceinline__ void load(int t0)
    {
        const int left = ch.tokens - t0;
        const char *kp = kbase + static_cast<int64_t>(t0) * p.kt * 2, *qp = qbase + static_cast<int64_t>(t0) * p.qt * 2;
        if (left >= TM) {
#pragma unroll
            for (int i = 0; i < kLoad; ++i) {
                nk[i] = *reinterpret_cast<const u32x4_a2 *>(kp + static_cast<int64_t>(i * kRows) * p.kt * 2 + koff);
                if constexpr (OUT)
                    nq[i] = *reinterpret_cast<const u32x4_a2 *>(qp + static_cast<int64_t>(i * kRows) * p.qt * 2 + qoff);
            }
        } else {
            const int t = here(tid / PK), c = here(tid % PK);
#pragma unroll
            for (int i = 0; i < kLoad; ++i) {
                const int in = t + kRows * i < left ? t + kRows * i : left - 1;
                nk[i] = *reinterpret_cast<const u32x4_a2 *>(kp + static_cast<uint32_t>(in) * static_cast<uint32_t>(2 * p.kt) + 16 * c);
                if constexpr (OUT)
                    nq[i] = *reinterpret_cast<const u32x4_a2 *>(qp + static_cast<uint32_t>(in) * static_cast<uint32_t>(2 * p.qt) + 16 * c);
            }
        }
        if (wave == kProducers - 1) {
            const int in = lane < left ? lane : left - 1;
            ng = gbase[static_cast<int64_t>(t0 + in) * p.gt];
            nb = bbase[static_cast<int64_t>(t0 + in) * p.bt];
        }
    }
    // And from there into LDS; rows past the end are zeros.
    __device__ __forceinline__ void store(LdsTile<K, TM> &to, int t0)
    {
        const int left = ch.tokens - t0, t = tid / PK, c = tid % PK;
        if (left < TM) {
#pragma unroll
            for (int i = 0; i < kLoad; ++i)
                if (t + kRows * i >= left)
                    nk[i] = nq[i] = u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kLoad; ++i) {
            *reinterpret_cast<u32x4_t *>(&to.k[t + kRows * i][8 * c]) = nk[i];
            if constexpr (OUT)
                *reinterpret_cast<u32x4_t *>(&to.q[t + kRows * i][8 * c]) = nq[i];
        }
        if (wave == kProducers - 1)
            gates(to, left);
    }
    // The decays and strengths of a tile, a token a lane.
    __device__ __forceinline__ void gates(LdsTile<K, TM> &to, int left)
    {
        const bool in = lane < left && lane < TM;
        float a = rate * softplus_f32(lo_f32(ng) + bias, dt_plain_above(1));
        a = a < kGone ? kGone : a;
        const double sum = prefix(in ? static_cast<double>(a) : 0.0, lane);
        const float hi = static_cast<float>(sum), lo = static_cast<float>(sum - static_cast<double>(hi));
        const float last_hi = __shfl(hi, 63), last_lo = __shfl(lo, 63);
        if (lane < TM) {
            to.g[0][lane] = hi;
            to.g[1][lane] = lo;
            to.decay[lane] = exp2_f32(hi + lo);
            to.left[lane] = exp2_f32((last_hi - hi) + (last_lo - lo));
            to.beta[lane] = in ? sigmoid_f32(lo_f32(nb)) : 0.0f;
            if (lane == 0)
                to.total = exp2_f32(last_hi + last_lo);
        }
    }
    // Blocks (b, c) of A and P: lane r is token 16 b + r, its registers tokens 16 c + 4 g + i before it.
    struct Products {
        f32x4_t kk, qk;
    };
    template <int b, int c>
    __device__ __forceinline__ Products products(const LdsTile<K, TM> &to)
    {
        const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
        Products y = {zero, zero};
#pragma unroll
        for (int e = 0; e < K / 32; ++e) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t *>(&to.k[16 * c + r][32 * e + 8 * g]);
            y.kk = mfma(x, b == c ? x : *reinterpret_cast<const u32x4_t *>(&to.k[16 * b + r][32 * e + 8 * g]), y.kk);
            if constexpr (OUT)
                y.qk = mfma(x, *reinterpret_cast<const u32x4_t *>(&to.q[16 * b + r][32 * e + 8 * g]), y.qk);
        }
        return y;
    }
    template <int b, int c>
    __device__ __forceinline__ void finish(LdsTile<K, TM> &to, const Products &raw)
    {
        const float hi = to.g[0][16 * b + r], lo = to.g[1][16 * b + r], strength = -to.beta[16 * b + r];
        const f32x4_t hj = *reinterpret_cast<const f32x4_t *>(&to.g[0][16 * c + 4 * g]);
        const f32x4_t lj = *reinterpret_cast<const f32x4_t *>(&to.g[1][16 * c + 4 * g]);
        f32x4_t x, y;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float f = exp2_f32((hi - hj[m]) + (lo - lj[m]));
            x[m] = b > c || 4 * g + m < r ? strength * f * raw.kk[m] : 0.0f;
            y[m] = b > c || 4 * g + m <= r ? f * raw.qk[m] : 0.0f;
        }
        *reinterpret_cast<f32x4_t *>(&to.a[a_block(b, c)][r][4 * g]) = x;
        if constexpr (!OUT)
            return;
        u32x2_t parts[2];
        split<2>(y, parts);
        *reinterpret_cast<u32x2_t *>(&to.p[0][p_block(b, c / 2)][r][8 * g + 4 * (c % 2)]) = parts[0];
        *reinterpret_cast<u32x2_t *>(&to.p[1][p_block(b, c / 2)][r][8 * g + 4 * (c % 2)]) = parts[1];
    }
    // Three blocks at once, their products interleaved.
    template <int b0, int c0, int b1, int c1, int b2, int c2>
    __device__ __forceinline__ void three(LdsTile<K, TM> &to)
    {
        const Products x = products<b0, c0>(to), y = products<b1, c1>(to), z = products<b2, c2>(to);
        finish<b0, c0>(to, x);
        finish<b1, c1>(to, y);
        finish<b2, c2>(to, z);
    }
    template <int b0, int c0, int b1, int c1>
    __device__ __forceinline__ void two(LdsTile<K, TM> &to)
    {
        const Products x = products<b0, c0>(to), y = products<b1, c1>(to);
        finish<b0, c0>(to, x);
        finish<b1, c1>(to, y);
    }
    // The inverses of the diagonal blocks I + A by forward substitution: lane (g, r)
    // has column r of block g, X_i = e_i - sum_(m < i) A_im X_m.
    __device__ __forceinline__ void invert(LdsTile<K, TM> &to)
    {
        const int bl = a_block(g < NB ? g : 0, g < NB ? g : 0);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = i == here(r) ? 1.0f : 0.0f;
#pragma unroll
            for (int m4 = 0; m4 < i; m4 += 4) {
                const f32x4_t a = *reinterpret_cast<const f32x4_t *>(&to.a[bl][i][m4]);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (m4 + m < i)
                        x[i] = fmaf(a[m], x[m4 + m], x[i]);  // -A is stored
            }
            if (i % 4 == 3)  // no more rows of A in registers at once
                asm volatile("" : "+v"(x[i]), "+v"(x[i - 1]), "+v"(x[i - 2]), "+v"(x[i - 3])::"memory");
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (g < NB) {
#pragma unroll
            for (int i = 0; i < 16; ++i) to.a[bl][i][r] = x[i];
        }
    }
    // A wave's share of them (the first wave inverts, the last one works out the gates).
    __device__ __forceinline__ void blocks(LdsTile<K, TM> &to)
    {
        static_assert(NB == 2 || NB == 4, "shares of two or four blocks");
        if constexpr (NB == 4) {
            if (wave == 0)
                two<0, 0, 1, 0>(to);
            else if (wave == 1)
                three<1, 1, 2, 0, 3, 0>(to);
            else if (wave == 2)
                three<2, 2, 2, 1, 3, 1>(to);
            else
                two<3, 2, 3, 3>(to);
        } else {
            if (wave == 0)
                finish<0, 0>(to, products<0, 0>(to));
            else if (wave == 1)
                finish<1, 0>(to, products<1, 0>(to));
            else if (wave == 2)
                finish<1, 1>(to, products<1, 1>(to));
        }
    }
    __device__ __forceinline__ void run(Shared<K, TM> &sh)
    {

        load(0);
        store(sh.tile[0], 0);
        if (TM < ch.tokens)
            load(TM);
        lds_barrier();
        blocks(sh.tile[0]);
        lds_barrier();
        int buf = 0;
        for (int t0 = 0; t0 < ch.tokens; t0 += TM, buf ^= 1) {
            // while the state waves read with K and Q of a tile, its inverses and the next one's rows ...
            if (wave == 0)
                invert(sh.tile[buf]);
            const bool more = t0 + TM < ch.tokens;
            if (more)
                store(sh.tile[buf ^ 1], t0 + TM);
            if (t0 + 2 * TM < ch.tokens)
                load(t0 + 2 * TM);
            lds_barrier();
            // ... and while they go through the tile, the next one's blocks
            if (more)
                blocks(sh.tile[buf ^ 1]);
            lds_barrier();
        }
    }
};

// A wave with 16 columns of the state.  OUT: the pass that writes out, from the
// states that the chains start with.  Otherwise the pass that forms every segment's
// own state, from zero (the first one's from the initial state), and, in K more
// columns without values, what it makes of each unit vector.
template <int K, int TM, bool OUT>
__device__ __forceinline__ void state_wave(const DeltaParams &p, const Chain &ch, Shared<K, TM> &sh, int lane, int wave)
{
    constexpr int KT = K / 16, KSTEP = K / 32, NB = TM / 16;  // state tiles; steps over k; blocks of tokens
    const int r = lane & 15, g = lane >> 4, col = ch.col0 + 16 * wave;
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};

    // the state: register i of tile 2 e + a is k = 32 e + 8 g + 4 a + i of column r
    f32x4_t s[KT];
    const auto place = [&](int t) { return 8 * g + 32 * (t / 2) + 4 * (t % 2); };
    const int64_t own = ((ch.n * p.H + ch.h) * p.V + col + r) * K;  // in the call's states
    const bool unit = !OUT && col >= p.V;
    const void *start = p.init_state;
    int kind = p.init_kind;
    int64_t from = own;
    if (OUT ? ch.several : ch.index > 0) {
        kind = OUT ? kFp32 : kNone;
        start = p.slabs;
        from = slab_row(p, ch.slab + ch.index, ch.h, col + r);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        s[t] = zero;
        if (kind == kFp32) {
            s[t] = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(start) + from + place(t));
        } else if (kind == kBf16) {
            const u32x2_t v = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(start) + from + place(t));
            s[t] = f32x4_t{lo_f32(v[0]), hi_f32(v[0]), lo_f32(v[1]), hi_f32(v[1])};
        }
        if (!OUT && ch.index == 0)  // for the pass to come, which may write the final state over the initial one
            *reinterpret_cast<f32x4_t *>(p.slabs + slab_row(p, ch.slab, ch.h, col + r) + place(t)) = s[t];
        if (unit) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][i] = place(t) + i == col + r - static_cast<int>(p.V) ? 1.0f : 0.0f;
        }
    }
    // The wave's own columns of V: half a row a lane, a tile ahead in registers.
    constexpr int kLoad = TM / 32;
    u32x4_t nv[kLoad];
    if (unit) {
#pragma unroll
        for (int i = 0; i < kLoad; ++i) nv[i] = u32x4_t{0, 0, 0, 0};
    }
    const char *vbase = reinterpret_cast<const char *>(p.v + ch.row * p.vb + static_cast<int64_t>(ch.begin) * p.vt + ch.h * p.V + col);
    const auto load = [&](int t0) {
        if (unit)
            return;
        const char *vp = vbase + static_cast<int64_t>(t0) * p.vt * 2;
        const int left = ch.tokens - t0, me = here(lane);
#pragma unroll
        for (int i = 0; i < kLoad; ++i) {
            const int t = me / 2 + 32 * i, in = t < left ? t : left - 1;
            nv[i] = *reinterpret_cast<const u32x4_a2 *>(vp + static_cast<uint32_t>(in) * static_cast<uint32_t>(2 * p.vt) + 16 * (me & 1));
        }
    };
    uint16_t *obase = p.out + ((ch.row * p.seqs.T + ch.begin) * p.H + ch.h) * p.V + col;
    const int64_t ostride = p.H * p.V;

    if (ch.tokens > 0) {
        load(0);
        lds_barrier();
        lds_barrier();
    }
    int buf = 0;
    for (int t0 = 0; t0 < ch.tokens; t0 += TM, buf ^= 1) {
        // places in the tile: a base for each pattern of lanes, and constants
        using T = LdsTile<K, TM>;
        const uint32_t base = lds_addr(&sh.tile[buf]), row = base + 2 * T::kPitch * r + 16 * g;
        const uint32_t ap = base + offsetof(T, a) + 4 * T::kAPitch * r + 16 * g;  // rows of A and P are equally long
        static_assert(4 * T::kAPitch == 2 * T::kPPitch, "");
        const uint32_t four = base + offsetof(T, decay) + 16 * g, one = base + offsetof(T, decay) + 4 * r;
        constexpr uint32_t kQ = offsetof(T, q), kABlock = sizeof(T::a[0]), kP = offsetof(T, p) - offsetof(T, a), kPart = sizeof(T::p[0]),
                           kPBlock = sizeof(T::p[0][0]), kBeta = offsetof(T, beta) - offsetof(T, decay),
                           kLeft = offsetof(T, left) - offsetof(T, decay), kTotal = offsetof(T, total) - offsetof(T, decay);
        const int left = ch.tokens - t0, me = here(lane);
#pragma unroll
        for (int i = 0; i < kLoad; ++i) {
            const int t = me / 2 + 32 * i;
            *reinterpret_cast<u32x4_t *>(&sh.v[wave][t][8 * (me & 1)]) = t < left ? nv[i] : u32x4_t{0, 0, 0, 0};
        }
        if (TM < left)
            load(t0 + TM);

        // K S and Q S: rows are tokens of K S, columns of (Q S)^T.  Accumulators in turn, so that none waits for its
        // own last product; rows of Q are asked for before the products of K's, and the next step's of K before those of Q
        f32x4_t u[NB], o[NB];
        u32x4_t kr[NB], qr[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) kr[b] = lds_load<u32x4_t>(row + 32 * T::kPitch * b);
#pragma unroll
        for (int e = 0; e < KSTEP; ++e) {
#pragma unroll
            for (int b = 0; OUT && b < NB; ++b) qr[b] = lds_load<u32x4_t>(row + kQ + 32 * T::kPitch * b + 64 * e);
            u32x2_t x[3], y[3];
            split<3>(s[2 * e], x);
            split<3>(s[2 * e + 1], y);
            const u32x4_t s0 = cat(x[0], y[0]), s1 = cat(x[1], y[1]), s2 = cat(x[2], y[2]);
#pragma unroll
            for (int b = 0; b < NB; ++b) u[b] = mfma(kr[b], s0, e > 0 ? u[b] : zero);
#pragma unroll
            for (int b = 0; b < NB; ++b) u[b] = mfma(kr[b], s1, u[b]);
#pragma unroll
            for (int b = 0; b < NB; ++b) u[b] = mfma(kr[b], s2, u[b]);
#pragma unroll
            for (int b = 0; e + 1 < KSTEP && b < NB; ++b) kr[b] = lds_load<u32x4_t>(row + 32 * T::kPitch * b + 64 * (e + 1));
#pragma unroll
            for (int b = 0; OUT && b < NB; ++b) o[b] = mfma(s0, qr[b], e > 0 ? o[b] : zero);
#pragma unroll
            for (int b = 0; OUT && b < NB; ++b) o[b] = mfma(s1, qr[b], o[b]);
        }
        // what the residual takes is there already
        const uint32_t vaddr = lds_addr(&sh.v[wave][here(lane) / 4][4 * (here(lane) & 3)]);  // 4 g + r / 4
        u32x2_t vr[NB];
        f32x4_t decay[NB], beta[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            vr[b] = lds_tr(vaddr + 512 * b);
            decay[b] = lds_load<f32x4_t>(four + 64 * b);
            beta[b] = lds_load<f32x4_t>(four + kBeta + 64 * b);
        }
        lds_barrier();

        // beta (V - 2^G K S)
        f32x4_t inv[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) inv[b] = lds_load<f32x4_t>(ap + kABlock * a_block(b, b));
        float fine[2] = {0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const f32x4_t v = {lo_f32(vr[b][0]), hi_f32(vr[b][0]), lo_f32(vr[b][1]), hi_f32(vr[b][1])};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[b][i] = beta[b][i] * fmaf(-decay[b][i], u[b][i], v[i]);
                fine[i & 1] = fmaf(u[b][i], 0.0f, fine[i & 1]);
            }
        }
        // The first token of column r that is odd; all from there on is taken out.
        int poison = TM;
        const auto clear = [&](int b) {
            const int g4 = here(4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[b][i] = 16 * b + g4 + i >= poison ? 0.0f : u[b][i];
        };
        const auto scrub = [&] {
            const int g4 = here(4 * g);
            int first = poison;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * b + g4 + i;
                    first = (__float_as_uint(u[b][i]) & 0x7fffffffu) >= kOddBits && t < first ? t : first;
                }
            const int other = __shfl_xor(first, 16), both = other < first ? other : first;
            const int far = __shfl_xor(both, 32);
            poison = far < both ? far : both;
#pragma unroll
            for (int b = 0; b < NB; ++b) clear(b);
        };
        bool poisoned = __any(fine[0] + fine[1] != 0.0f);
        if (poisoned)
            scrub();
        // U, block by block
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (poisoned)
                clear(b);  // rows of A may not be finite, either
            u[b] = mfma_f32(inv[b], u[b], zero);
            // step by step over the blocks below, so that none waits for its own last product
            f32x4_t below[NB];
#pragma unroll
            for (int c = b + 1; c < NB; ++c) below[c] = lds_load<f32x4_t>(ap + kABlock * a_block(c, b));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = b + 1; c < NB; ++c) u[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(below[c][i], u[b][i], u[c], 0, 0, 0);
        }
        u32x2_t up[NB][2];
        uint32_t most = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            split<2>(u[b], up[b]);
            most = max_bf16(max_bf16(most, up[b][0][0]), up[b][0][1]);
        }
        if (__any((most & 0xffffu) >= 0x7f80u || most >= 0x7f800000u)) {
            scrub();
            poisoned = true;
#pragma unroll
            for (int b = 0; b < NB; ++b) split<2>(u[b], up[b]);
        }

        if constexpr (OUT) {
            // out
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                o[b] *= lds_load<float>(one + 64 * b);
#pragma unroll
                for (int e = 0; 2 * e + 1 <= b; ++e) {
                    const uint32_t at = ap + kP + kPBlock * p_block(b, e);
                    const u32x4_t p0 = lds_load<u32x4_t>(at), p1 = lds_load<u32x4_t>(at + kPart);
                    const u32x4_t u0 = cat(up[2 * e][0], up[2 * e + 1][0]), u1 = cat(up[2 * e][1], up[2 * e + 1][1]);
                    o[b] = mfma(u0, p0, o[b]);
                    o[b] = mfma(u1, p0, o[b]);
                    o[b] = mfma(u0, p1, o[b]);
                }
                if (b % 2 == 0) {
                    // the block that is left, in a sum of its own: a product over 16 slots right behind one over 32
                    // on the same accumulator, which the compiler does not keep apart, gave wrong sums
                    const uint32_t at = ap + kP + kPBlock * p_block(b, b / 2);
                    const u32x2_t p0 = lds_load<u32x2_t>(at), p1 = lds_load<u32x2_t>(at + kPart);
                    f32x4_t x = mfma16(up[b][0], p0, zero);
                    x = mfma16(up[b][1], p0, x);
                    x = mfma16(up[b][0], p1, x);
                    o[b] += x;
                }
                o[b] *= p.scale;
            }
            if (poisoned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = __shfl(poison, here(4 * g) + i);
#pragma unroll
                    for (int b = 0; b < NB; ++b) o[b][i] = 16 * b + here(r) >= from ? __builtin_nanf("") : o[b][i];
                }
            }
            uint16_t *op = obase + (t0 + here(r)) * ostride + here(4 * g);
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (16 * b + r < left)
                    *reinterpret_cast<u32x2_t *>(op + 16 * b * ostride) =
                        u32x2_t{pack_bf16x2(o[b][0], o[b][1]), pack_bf16x2(o[b][2], o[b][3])};
        }
        fence();

        // the state
        u32x2_t w[NB][3];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            split<3>(u[b] * lds_load<f32x4_t>(four + kLeft + 64 * b), w[b]);
        }
        const float total = lds_load<float>(base + offsetof(T, decay) + kTotal);
        const uint32_t kaddr = base + 2 * T::kPitch * (here(lane) / 4) + 16 * (here(lane) & 3);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            s[t] *= total;
#pragma unroll
            for (int e = 0; e < NB / 2; ++e) {
                const uint32_t at = kaddr + 2 * (32 * (t / 2) + 4 * (t % 2)) + 64 * T::kPitch * e;
                const u32x4_t kr = cat(lds_tr(at), lds_tr(at + 32 * T::kPitch));
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
        lds_barrier();
    }

    if (OUT && (!p.final_state || !ch.last))
        return;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        if (!OUT)
            *reinterpret_cast<f32x4_t *>(p.slabs + slab_row(p, ch.slab + ch.index + 1, ch.h, col + r) + place(t)) = s[t];
        else if (p.final_kind == kFp32)
            *reinterpret_cast<f32x4_t *>(static_cast<float *>(p.final_state) + own + place(t)) = s[t];
        else
            *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(p.final_state) + own + place(t)) =
                u32x2_t{pack_bf16x2(s[t][0], s[t][1]), pack_bf16x2(s[t][2], s[t][3])};
    }
}

template <int K, int TM, bool OUT>
__global__ __launch_bounds__(kThreads) void delta_chunk_kernel(DeltaParams p, int vblocks, int columns)
{
    __shared__ __align__(16) Shared<K, TM> sh;
    static_assert(sizeof(sh) <= 160 * 1024, "LDS of a compute unit");
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Chain ch = find_chain(p, static_cast<int>(OUT ? p.V : p.V + p.K), vblocks, columns);
    // own states: of all segments but a sequence's last; what the first one makes of unit vectors is not asked
    if (!ch.valid || (!OUT && (ch.last || (ch.index == 0 && ch.col0 >= p.V))))
        return;
    if (wave >= kStateWaves) {
        if (ch.tokens > 0) {
            Producer<K, TM, OUT> producer(p, ch, tid - 64 * kStateWaves, wave - kStateWaves);
            producer.run(sh);
        }
    } else if (16 * wave < ch.width && (OUT || ch.index > 0 || ch.col0 + 16 * wave < p.V)) {
        state_wave<K, TM, OUT>(p, ch, sh, tid & 63, wave);
    } else {
        // a wave without columns keeps the others' count of barriers: two a tile and two before
        for (int t0 = -TM; t0 < ch.tokens && ch.tokens > 0; t0 += TM) {
            lds_barrier();
            lds_barrier();
        }
    }
}

// The states that segments start with, one after the other: the end of segment j is
// its own state plus what it makes of the end of the one before,
//   S_j[v, :] <- S_j[v, :] + sum_k S_(j-1)[v, k] M_j[k, :]
// in fp32 throughout.  A workgroup takes 16 rows v of a chain, a wave 16 of its K
// columns, in v_mfma_f32_16x16x4_f32: rows of the result are columns of M, and the
// state before, shared in LDS, is the right factor.
template <int K>
__global__ __launch_bounds__(4 * K) void delta_join_kernel(DeltaParams p)
{
    constexpr int KT = K / 16;
    __shared__ __align__(16) float before[2][16][K + 4];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t vblocks = static_cast<uint32_t>(p.V / 16), chain = blockIdx.x / vblocks, v0 = 16 * (blockIdx.x - chain * vblocks);
    const uint32_t n = chain / static_cast<uint32_t>(p.H);
    const int64_t h = chain - n * static_cast<uint32_t>(p.H);
    const uint32_t seg = static_cast<uint32_t>(p.seg), begin = p.seqs.cu ? clamp_offset(p.seqs, n) : 0,
                   end = p.seqs.cu ? clamp_offset(p.seqs, n + 1) : static_cast<uint32_t>(p.seqs.T);
    const uint32_t count = end > begin ? (end - begin + seg - 1) / seg : 0;
    if (count < 3)
        return;
    const int64_t first = p.map.mul * (begin / seg) + p.map.add * n;
    const auto at = [&](uint32_t j) { return reinterpret_cast<f32x4_t *>(p.slabs + slab_row(p, first + j, h, v0 + r) + 16 * wave + 4 * g); };
    // M a step ahead, where the registers hold it
    constexpr bool kAhead = K <= 128;
    float m[kAhead ? KT : 1][4];
    const auto map = [&](uint32_t j) { return p.slabs + slab_row(p, first + j, h, p.V + 4 * g) + 16 * wave + r; };
    const auto load = [&](uint32_t j) {
        const float *src = map(j);
#pragma unroll
        for (int t = 0; t < (kAhead ? KT : 0); ++t, src += 16 * K)
#pragma unroll
            for (int i = 0; i < 4; ++i) m[t][i] = src[i * K];
    };
    f32x4_t s = *at(1), next = *at(2);
    load(2);
    int buf = 0;
    for (uint32_t j = 2; j < count; ++j, buf ^= 1) {
        *reinterpret_cast<f32x4_t *>(&before[buf][r][16 * wave + 4 * g]) = s;
        lds_barrier();
        s = next;
        const float *src = map(j);
#pragma unroll(kAhead ? KT : 2)
        for (int t = 0; t < KT; ++t, src += 16 * K) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t *>(&before[buf][r][16 * t + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x4f32(kAhead ? m[kAhead ? t : 0][i] : src[i * K], x[i], s, 0, 0, 0);
        }
        if (j + 1 < count) {
            load(j + 1);
            next = *at(j + 1);
        }
        *at(j) = s;
    }
}

// Columns a workgroup takes at most.  Its tile takes 14000 cycles with eight state
// waves, two a SIMD, and 7000 to 9000 with one to four, so few chains are spread:
// as thinly as 256 workgroups, one a compute unit, allow.  Of
// one of 8191 tokens with 12 heads of 64 x 96, uncut, 128 columns take 567 us, 48 417, 32
// 404 and 16 391; of 8 x 16384 with 32 heads of 128 128 take 1690, 64 2070.  Of packed
// sequences of unequal lengths 512 with 64 columns: the second half starts where short
// ones end (19595 tokens in 8 sequences with 32 heads 128 take 430, 64 396 and 32 638; 16384
// in 3 with 60 heads 128 630 to 970, 64 520 to 640), but with fewer columns, which save
// nothing more, 256 (2 with 40 heads: 64 560 to 840, 32 670 to 810; 4 with 32
// 320 to 540, 32 510 to 530).
int columns_of(int64_t chains, int64_t all, bool unequal)
{
    int columns = 16;
    while (columns < kColumns && columns < all &&
           chains * ((all + columns - 1) / columns) > (unequal && columns >= kColumns / 2 ? 512 : 256))
        columns *= 2;
    return columns < all ? columns : static_cast<int>(all);
}

template <int K, int TM, bool OUT>
hipError_t launch_pass(const DeltaParams &p, int64_t slots, hipStream_t stream)
{
    const int64_t all = OUT ? p.V : p.V + p.K;
    const int most = columns_of(slots * p.H, all, p.seqs.cu && p.seqs.N > 1 && p.seg == 0);
    const int64_t vblocks = (all + most - 1) / most, blocks = slots * p.H * vblocks;
    const int columns = static_cast<int>((all / 16 + vblocks - 1) / vblocks * 16);  // as evenly as waves allow
    if (!grid_fits(blocks, kThreads))
        return hipErrorInvalidConfiguration;
    delta_chunk_kernel<K, TM, OUT><<<dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream>>>(p, static_cast<int>(vblocks), columns);
    return hipGetLastError();
}

template <int K, int TM>
hipError_t launch(const DeltaParams &p, hipStream_t stream)
{
    if (p.seg == 0)
        return launch_pass<K, TM, true>(p, p.seqs.N, stream);
    const int64_t slots = tile_slots(p.seqs, p.seg), joins = p.seqs.N * p.H * (p.V / 16);
    if (!grid_fits(joins, 4 * K) || !grid_fits(slots * p.H * ((p.V + p.K + 15) / 16), kThreads))
        return hipErrorInvalidConfiguration;  // before anything is enqueued
    hipError_t e = launch_pass<K, TM, false>(p, slots, stream);
    if (e != hipSuccess)
        return e;
    delta_join_kernel<K><<<dim3(static_cast<uint32_t>(joins)), dim3(4 * K), 0, stream>>>(p);
    e = hipGetLastError();
    return e != hipSuccess ? e : launch_pass<K, TM, true>(p, slots, stream);
}

}  // namespace

hipError_t launch_delta_chunk(const DeltaParams &p, hipStream_t stream)
{
    switch (p.K) {
    case 64: return launch<64, 64>(p, stream);
    case 128: return launch<128, 64>(p, stream);
    case 256: return launch<256, 32>(p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace layer
}  // namespace kda
