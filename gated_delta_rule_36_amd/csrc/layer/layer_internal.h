// Internal interface between the C-ABI front end of the layer operators
// (layer_api.cpp) and their HIP kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace kda {
namespace layer {

// Element kinds of parameters, residual streams and states (kda_dtype values).
enum Kind : int { kNone = 0, kBf16 = 1, kFp32 = 2 };
enum Act : int { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

constexpr int64_t kMaxTaps = 8;         // W of the convolution
constexpr int64_t kMaxNormSize = 16384; // elements one norm spans

// Sequences: a batch (cu == nullptr: N sequences of T tokens, one per batch
// row) or packed along the token axis of one row.
struct Seqs {
    const int64_t *cu;
    int64_t N, T;
};

// Work slots for tiles of len tokens (see find_tile in layer_device.h).
inline int64_t tile_slots(const Seqs &s, int64_t len)
{
    if (s.cu)
        return s.T / len + s.N;
    return s.N * (s.T > 0 ? (s.T + len - 1) / len : 1);
}

// State slabs for sequences of more than one segment of len tokens, one a
// segment; a sequence of one segment takes its state where it lies, so that many
// short ones need no more than T / len allow.  The slabs of sequence n, over
// tokens [a, b), start at mul floor(a / len) + add n.  In a batch each has as
// many as segments.  Of packed ones, count = ceil((b - a) / len) is at most
// floor(b / len) - floor(a / len) + 1, which leaves room with (1, 1); and from two
// segments on count <= 2 (count - 1), which leaves room with (2, 0).  All slabs
// are below the total for any offsets 0 <= a <= b <= T, in order or not.
struct SlabMap {
    int64_t mul, add, slabs;
};
inline SlabMap slab_map(const Seqs &s, int64_t len)
{
    if (!s.cu) {
        const int64_t per = (s.T + len - 1) / len;
        return {0, per, per > 1 ? s.N * per : 0};
    }
    const int64_t whole = s.T / len;
    return s.N < whole ? SlabMap{1, 1, whole + s.N} : SlabMap{2, 0, 2 * whole};
}

// Whether a grid of one dimension takes this many workgroups: a launch counts
// its threads in 32 bits.  Launches that do not fit return
// hipErrorInvalidConfiguration.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= UINT32_MAX / threads; }

// A norm's eps, and times 2^188 and 2^-160 for rows whose squares fp32 does not
// hold (see norm_shift in layer_device.h).
struct NormEps {
    float plain, up, down;
};
inline NormEps norm_eps(double eps)
{
    return {static_cast<float>(eps), static_cast<float>(eps * 0x1p188), static_cast<float>(eps * 0x1p-160)};
}

struct ConvParams {
    const uint16_t *x;
    int64_t xb, xt;  // element strides of batch row and token
    const void *weight, *bias;
    int weight_kind;
    uint16_t *out;
    const void *init_state;
    void *final_state;
    int init_kind, final_kind;
    Seqs seqs;
    int64_t D;
    int act, l2norm;
    NormEps l2eps;
};
hipError_t launch_conv(const ConvParams &p, int W, hipStream_t stream);

struct GatedParams {
    const uint16_t *x, *gate;  // gate may be nullptr
    int64_t xr, gr;            // element strides of a row
    const void *weight;        // [D]
    int weight_kind;
    uint16_t *out;
    int64_t rows, D, group;
    int act, gate_first;
    NormEps eps;
};
hipError_t launch_gated_norm(const GatedParams &p, hipStream_t stream);

struct ResidParams {
    const uint16_t *x;
    int64_t xr;
    const void *residual;  // or nullptr
    void *residual_out;    // or nullptr
    int residual_kind, residual_out_kind;
    const void *post_weight, *weight;  // or nullptr
    int post_kind, weight_kind;
    const void *gate;  // or nullptr; row r reads gate row r / gate_period
    int gate_kind;
    int64_t gr, gate_period;
    uint16_t *out;  // or nullptr
    int64_t rows, D;
    float residual_scale, block_scale;
    NormEps eps;
};
hipError_t launch_residual_norm(const ResidParams &p, hipStream_t stream);

struct SsmParams {
    const uint16_t *x, *dt, *b, *c, *z;  // z may be nullptr
    int64_t xb, xt, db, dtt, bb, bt, cb, ct, zb, zt;  // element strides of batch row and token
    uint16_t *out;
    const float *A_log, *D, *dt_bias;  // D, dt_bias may be nullptr
    const void *init_state;
    void *final_state;
    int init_kind, final_kind;
    Seqs seqs;
    int64_t H, P, G, N;
    int softplus;
    // chunked kernel: tokens a segment; if a sequence can have more than one, the
    // slabs (see slab_map): a state [H,P,N] and log decays [H] each (else nullptr)
    int64_t seg;
    SlabMap map;
    float *slabs, *logs;
};
// Tokens per chunk of the chunked kernel; segments are multiples of it.
constexpr int64_t kSsmChunk = 32;
// Calls without cu_seqlens of at most this many tokens take the token
// recurrence.  32 heads of 64 x 128, in us, by it (by the chunked kernel): 64 rows
// of 8 tokens 41 (47), of 9 43 (47), of 12 52 (47), of 16 63 (47); 8 rows of 8 11
// (20), of 16 16 (20); one row of 8 9 (18), of 16 14 (19).  64 heads of 64 x 64: 64
// rows of 8 43 (57), of 9 47 (58), of 12 58 (57); 8 rows of 12 13 (15), of 16 17
// (15).  So at 8 it is the faster one for every batch measured; between 9 and 16
// that depends on the batch, and the limit goes by tokens alone, so that a row's
// roundings do not depend on how many others the call has.
constexpr int64_t kSsmRecurrentMaxTokens = 8;

hipError_t launch_ssm_recurrent(const SsmParams &p, hipStream_t stream);
hipError_t launch_ssm_chunk(const SsmParams &p, hipStream_t stream);
// Waves of a workgroup of the chunked kernel, and columns a wave takes.
constexpr int64_t kSsmWaves = 8, kSsmColumns = 32;
// Tokens a call: the chunked kernel counts a segment's in 32 bits with sign, up to
// two tiles (of two chunks) past its end.
constexpr int64_t kSsmMaxTokens = INT32_MAX - 4 * kSsmChunk;
// Token strides (elements) whose lane offsets stay within 32 bits of bytes: a
// wave loads up to 16 rows of x, b or c from one base, and 32 of z.
constexpr int64_t kSsmMaxStride = int64_t(1) << 27, kSsmMaxZStride = int64_t(1) << 26;

struct DeltaParams {
    const uint16_t *q, *k, *v, *g, *beta;
    int64_t qb, qt, kb, kt, vb, vt, gb, gt, bb, bt;  // element strides of batch row and token
    uint16_t *out;
    const float *A_log, *dt_bias;  // dt_bias may be nullptr
    const void *init_state;
    void *final_state;
    int init_kind, final_kind;
    Seqs seqs;
    int64_t H, G, K, V;
    float scale;
    // the chunked kernel: tokens a segment, 0 for whole sequences; of segments the
    // slabs [H, V + K, K] (see slab_map; nullptr where every sequence is one segment)
    int64_t seg;
    SlabMap map;
    float *slabs;
};
// Segments are multiples of this many tokens.
constexpr int64_t kDeltaTile = 64;
hipError_t launch_delta_recurrent(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_chunk(const DeltaParams &p, hipStream_t stream);
constexpr int64_t kDeltaMaxV = 512;
// Tokens a call: places are counted in 32 bits with sign, up to two tiles past
// a sequence's end.  Token strides (elements) whose 64 rows of a tile stay
// within 32 bits of bytes.
constexpr int64_t kDeltaMaxTokens = INT32_MAX - 128, kDeltaMaxStride = int64_t(1) << 24;
// Sequences of at most this many tokens take the token recurrence.
constexpr int64_t kDeltaRecurrentMaxTokens = 8;

// Channels of a head that the rotation kernels take.
constexpr int64_t kMaxHeadChannels = 512;

// A paged cache: element strides of page, token and head.
struct CacheStrides {
    int64_t page, token, head;
};

// Norm and rotation of the rows of a token: `first` heads of x and then `second`
// of y.  For the append, x are the keys and y the values, which go as they are
// to `slots` of two caches.
struct RotaryParams {
    const uint16_t *x, *y;
    int64_t xb, xt, yb, yt;  // element strides of batch row and token
    uint16_t *x_out, *y_out;
    const int64_t *positions;  // or nullptr: no rotation
    const float *inv_freq;
    const void *x_weight, *y_weight;  // or nullptr: no norm
    int x_kind, y_kind;
    int64_t B, T;
    int first, second, D, R, interleaved;
    NormEps eps;
    float scale;
    // the append
    const int64_t *slots;
    int64_t slot_count, page_size;
    CacheStrides xc, yc;
};
hipError_t launch_rotary(const RotaryParams &p, hipStream_t stream);

struct AttentionParams {
    const uint16_t *q, *k, *v;
    int64_t qr;
    CacheStrides ks, vs;
    const int32_t *table, *lengths;
    int64_t table_stride;
    uint16_t *out;
    float *lse;  // or nullptr
    int64_t N, Hq, Hk, D, pages, width, window;
    uint32_t page_size, page_mul;  // t / page_size = umulhi(t, page_mul) >> page_shift for t < 2^31 (page_size > 1)
    int page_shift;
    int64_t splits;
    int chunk;    // tokens a split
    bool shared;  // a workgroup's waves share a split
    float scale;
    // of several splits: their unnormalised outputs [N, Hq, splits, D] and
    // (maximum, sum) [N, Hq, splits, 2]
    float *part, *stats;
};
constexpr int64_t kAttentionMaxD = 256;
// Query heads of a key head that a wave takes, and tokens at a time.
constexpr int64_t kAttentionRows = 16, kAttentionTile = 32;
hipError_t launch_paged_attention(const AttentionParams &p, hipStream_t stream);

}  // namespace layer
}  // namespace kda
