// C-ABI front end of the layer operators: argument checks on the host, then
// the hand-off to the kernels.  Nothing here touches device memory.
#include <algorithm>
#include <cstdint>

#include "layer_checks.h"

namespace {

using namespace kda::layer;

constexpr int64_t kMaxChannels = int64_t(1) << 24;

}  // namespace

extern "C" kda_status kda_short_conv(const kda_conv_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_conv_args &a = *args;
    if (a.reserved != 0 || (a.activation != KDA_ACT_NONE && a.activation != KDA_ACT_SILU))
        return KDA_ERR_OPTION;
    if (a.W < 1 || a.W > kda::layer::kMaxTaps || a.D < 1 || a.D > kMaxChannels ||
        (a.l2norm != 0 && a.l2norm != 64 && a.l2norm != 128 && a.l2norm != 256) ||
        (a.l2norm != 0 && a.D % a.l2norm != 0))
        return KDA_ERR_SHAPE;
    if (a.l2norm != 0 && !valid_eps(a.l2norm_eps))
        return KDA_ERR_SCALE;
    if (!bf16_or_fp32(a.weight_dtype))
        return KDA_ERR_DTYPE;
    kda::layer::ConvParams p = {};
    kda_status st = check_seqs(a.cu_seqlens, a.num_seqs, a.B, a.T, &p.seqs);
    if (st == KDA_OK)
        st = check_states(a.initial_state, a.initial_state_dtype, a.final_state, a.final_state_dtype);
    if (st != KDA_OK)
        return st;
    int64_t tokens, out_bytes, state, in_bytes;
    if (!mul_ok(a.B, a.T, &tokens) || !mul_ok(tokens, 2 * a.D, &out_bytes) ||
        !mul_ok(p.seqs.N, 4 * (a.W - 1) * a.D, &state))
        return KDA_ERR_SIZE;
    if (!extent(a.B, a.x_stride_b, a.T, a.x_stride_t, a.D, 2, &in_bytes))
        return KDA_ERR_STRIDE;
    if ((tokens > 0 && (!a.x || !a.out)) || !a.weight)
        return KDA_ERR_NULL_POINTER;
    const int64_t we = bytes_of(a.weight_dtype);
    const Span sx = span(a.x, in_bytes), sw = span(a.weight, a.D * a.W * we), sb = span(a.bias, a.D * we),
               sc = span(a.cu_seqlens, a.cu_seqlens ? (p.seqs.N + 1) * 8 : 0), so = span(a.out, out_bytes),
               si = span(a.initial_state, a.initial_state ? state / 4 * bytes_of(a.initial_state_dtype) : 0),
               sf = span(a.final_state, a.final_state ? state / 4 * bytes_of(a.final_state_dtype) : 0);
    if (any_overlap(so, {sx, sw, sb, sc, si, sf}) || any_overlap(sf, {sx, sw, sb, sc}) ||
        (sf.overlaps(si) && a.final_state != a.initial_state))
        return KDA_ERR_ALIAS;
    if (misaligned(a.x, 2) || misaligned(a.out, 16) || misaligned(a.weight, we) || misaligned(a.bias, we) ||
        misaligned(a.initial_state, 16) || misaligned(a.final_state, 16) || misaligned(a.cu_seqlens, 8))
        return KDA_ERR_ALIGNMENT;
    p.x = static_cast<const uint16_t *>(a.x);
    p.xb = a.x_stride_b;
    p.xt = a.x_stride_t;
    p.weight = a.weight;
    p.bias = a.bias;
    p.weight_kind = a.weight_dtype;
    p.out = static_cast<uint16_t *>(a.out);
    p.init_state = a.initial_state;
    p.final_state = a.final_state;
    p.init_kind = a.initial_state_dtype;
    p.final_kind = a.final_state_dtype;
    p.D = a.D;
    p.act = a.activation;
    p.l2norm = static_cast<int>(a.l2norm);
    p.l2eps = kda::layer::norm_eps(a.l2norm_eps);
    if (p.seqs.N == 0 || (tokens == 0 && !a.final_state))
        return KDA_OK;
    return launched(kda::layer::launch_conv(p, static_cast<int>(a.W), static_cast<hipStream_t>(stream)));
}

namespace {

// Sizes of a scan call: KDA_OK and the sequences, or what is wrong.
kda_status check_ssm_sizes(const kda_ssm_args &a, Seqs *s)
{
    if (a.P < 32 || a.P > 256 || a.P % 32 != 0 || (a.N != 32 && a.N != 64 && a.N != 128 && a.N != 256) ||
        a.seg_tokens < 0 || a.seg_tokens % kda::layer::kSsmChunk != 0)
        return KDA_ERR_SHAPE;
    if (a.H < 1 || a.H > 65536 || a.T > kda::layer::kSsmMaxTokens)
        return KDA_ERR_SIZE;
    if (a.G < 1 || a.H % a.G != 0)
        return KDA_ERR_SHAPE;
    const kda_status st = check_seqs(a.cu_seqlens, a.num_seqs, a.B, a.T, s);
    int64_t rows, n;
    if (st == KDA_OK && (!mul_ok(a.B, a.T, &rows) || !mul_ok(rows, a.H * a.P * 2, &n) ||
                         !mul_ok(s->N, a.H * a.P * a.N * 4, &n) || s->N * a.H > INT32_MAX))
        return KDA_ERR_SIZE;
    return st;
}

}  // namespace

namespace {

// How a scan call with valid sizes runs.
struct SsmPlan {
    bool recurrent = false;
    int64_t seg = 0;              // tokens a segment (chunked kernel)
    kda::layer::SlabMap map = {};  // no slabs without segments
    int64_t slab = 0;              // floats a slab
    int64_t bytes = 0;             // workspace
};

// Calls without cu_seqlens of up to kSsmRecurrentMaxTokens tokens: the token
// recurrence.  The others: as many segments as give every compute unit of 256
// one workgroup and no more (one fits a unit, and a second round costs as much
// as the first: 4 rows of 4096 tokens, 32 heads of 64 x 128, take 139 us in 8
// segments a row, 170 in 16, 210 in 4 and 585 whole), of whole tiles of the
// kernel (2048 tokens of 8 heads take 37 us in segments of one tile, 45 of two,
// 63 of four).  A batch is cut into equal parts.
// The lengths of packed sequences are not known here: each is taken to end half a
// segment early, and half the segments are kept however many sequences there
// are, for one of them may be long.  Of five random sets of lengths each, 32
// heads of 64 x 128, us by this rule (in segments of 256 / 768 / 2048 tokens):
//   2 sequences of 8192 tokens in all   95 - 98 (100 - 129 / 159 - 162 / 368 - 390)
//   8 of 19595                          175 - 184 (220 - 230 / 182 - 187 / 388 - 405)
//   32 of 16384                         145 - 166 (194 - 205 / 178 - 222 / 137 - 166)
//   128 of 16384                        207 - 224 (223 - 231 / 209 - 220 / 210 - 220)
// It loses where short ends add up to a segment more than there is room for: 8 of
// 19595 tokens in 33 segments take 271 us, and would 182 in those of 768.
// False if the workspace overflows.
bool ssm_plan(const kda_ssm_args &a, const Seqs &s, SsmPlan *plan)
{
    constexpr int64_t kTarget = 256, c = kda::layer::kSsmChunk, kTile = 2 * c;
    if (!s.cu && s.T <= kda::layer::kSsmRecurrentMaxTokens) {
        plan->recurrent = true;
        return true;
    }
    const int64_t columns = kda::layer::kSsmWaves * kda::layer::kSsmColumns;
    const int64_t blocks = a.G * ((a.H / a.G * a.P + columns - 1) / columns);
    const int64_t longest = s.T > c ? (s.T + c - 1) / c * c : c;
    int64_t seg = a.seg_tokens;
    if (seg == 0) {
        int64_t parts = kTarget / blocks;  // segments in all
        if (s.cu)
            parts = std::max(parts / 2, parts - s.N / 2);
        else
            parts /= s.N;
        if (parts < 1)
            parts = 1;
        seg = ((s.T + parts - 1) / parts + kTile - 1) / kTile * kTile;
        if (seg == 0)
            seg = kTile;
    }
    plan->seg = seg < longest ? seg : longest;
    if (plan->seg >= longest)
        return true;
    plan->map = kda::layer::slab_map(s, plan->seg);
    plan->slab = a.H * a.P * a.N;
    int64_t n;
    return mul_ok(plan->map.slabs, 4 * (plan->slab + a.H), &n) && add_ok(n, 15, &plan->bytes) && (plan->bytes &= ~int64_t(15)) >= 0;
}

}  // namespace

extern "C" int64_t kda_ssm_workspace_bytes(const kda_ssm_args *args)
{
    Seqs s;
    SsmPlan plan;
    if (!args || check_ssm_sizes(*args, &s) != KDA_OK || !ssm_plan(*args, s, &plan))
        return -1;
    return plan.bytes;
}

extern "C" kda_status kda_ssm_fwd(const kda_ssm_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_ssm_args &a = *args;
    if (a.reserved != 0 || !flag(a.softplus))
        return KDA_ERR_OPTION;
    kda::layer::SsmParams p = {};
    kda_status st = check_ssm_sizes(a, &p.seqs);
    if (st == KDA_OK)
        st = check_states(a.initial_state, a.initial_state_dtype, a.final_state, a.final_state_dtype);
    if (st != KDA_OK)
        return st;
    SsmPlan plan;
    if (!ssm_plan(a, p.seqs, &plan))
        return KDA_ERR_SIZE;
    const int64_t tokens = a.B * a.T, inner = a.H * a.P, state = p.seqs.N * inner * a.N;
    int64_t nx, nd, nb, nc, nz;
    if (!extent(a.B, a.x_stride_b, a.T, a.x_stride_t, inner, 2, &nx) ||
        !extent(a.B, a.dt_stride_b, a.T, a.dt_stride_t, a.H, 2, &nd) ||
        !extent(a.B, a.b_stride_b, a.T, a.b_stride_t, a.G * a.N, 2, &nb) ||
        !extent(a.B, a.c_stride_b, a.T, a.c_stride_t, a.G * a.N, 2, &nc) ||
        !extent(a.B, a.z_stride_b, a.T, a.z_stride_t, inner, 2, &nz))
        return KDA_ERR_STRIDE;
    if (!plan.recurrent && a.T > 1 &&
        (a.x_stride_t > kda::layer::kSsmMaxStride || a.b_stride_t > kda::layer::kSsmMaxStride ||
         a.c_stride_t > kda::layer::kSsmMaxStride || (a.z && a.z_stride_t > kda::layer::kSsmMaxZStride)))
        return KDA_ERR_STRIDE;
    if ((tokens > 0 && (!a.x || !a.dt || !a.b || !a.c || !a.out)) || !a.A_log)
        return KDA_ERR_NULL_POINTER;
    const Span sx = span(a.x, nx), sd = span(a.dt, nd), sb = span(a.b, nb), sc = span(a.c, nc), sz = span(a.z, nz),
               sA = span(a.A_log, a.H * 4), sD = span(a.D, a.H * 4), st_ = span(a.dt_bias, a.H * 4),
               su = span(a.cu_seqlens, a.cu_seqlens ? (p.seqs.N + 1) * 8 : 0), so = span(a.out, tokens * inner * 2),
               si = span(a.initial_state, a.initial_state ? state * bytes_of(a.initial_state_dtype) : 0),
               sf = span(a.final_state, a.final_state ? state * bytes_of(a.final_state_dtype) : 0);
    if (any_overlap(so, {sx, sd, sb, sc, sz, sA, sD, st_, su, si, sf}) ||
        any_overlap(sf, {sx, sd, sb, sc, sz, sA, sD, st_, su}) ||
        (sf.overlaps(si) && a.final_state != a.initial_state))
        return KDA_ERR_ALIAS;
    if (misaligned(a.x, 2) || misaligned(a.dt, 2) || misaligned(a.b, 2) || misaligned(a.c, 2) || misaligned(a.z, 2) ||
        misaligned(a.out, 16) || misaligned(a.initial_state, 16) || misaligned(a.final_state, 16) ||
        misaligned(a.A_log, 4) || misaligned(a.D, 4) || misaligned(a.dt_bias, 4) || misaligned(a.cu_seqlens, 8))
        return KDA_ERR_ALIGNMENT;
    if (plan.bytes > 0) {
        if (!a.workspace || a.workspace_bytes < plan.bytes || misaligned(a.workspace, 16) ||
            any_overlap(span(a.workspace, plan.bytes), {sx, sd, sb, sc, sz, sA, sD, st_, su, so, si, sf}))
            return KDA_ERR_WORKSPACE;
    }
    p.x = static_cast<const uint16_t *>(a.x);
    p.dt = static_cast<const uint16_t *>(a.dt);
    p.b = static_cast<const uint16_t *>(a.b);
    p.c = static_cast<const uint16_t *>(a.c);
    p.z = static_cast<const uint16_t *>(a.z);
    p.out = static_cast<uint16_t *>(a.out);
    p.xb = a.x_stride_b;
    p.xt = a.x_stride_t;
    p.db = a.dt_stride_b;
    p.dtt = a.dt_stride_t;
    p.bb = a.b_stride_b;
    p.bt = a.b_stride_t;
    p.cb = a.c_stride_b;
    p.ct = a.c_stride_t;
    p.zb = a.z_stride_b;
    p.zt = a.z_stride_t;
    p.A_log = a.A_log;
    p.D = a.D;
    p.dt_bias = a.dt_bias;
    p.init_state = a.initial_state;
    p.final_state = a.final_state;
    p.init_kind = a.initial_state ? a.initial_state_dtype : KDA_DTYPE_NONE;
    p.final_kind = a.final_state ? a.final_state_dtype : KDA_DTYPE_NONE;
    p.H = a.H;
    p.P = a.P;
    p.G = a.G;
    p.N = a.N;
    p.softplus = a.softplus;
    if (p.seqs.N == 0 || (tokens == 0 && !a.final_state))
        return KDA_OK;
    if (plan.recurrent)
        return launched(kda::layer::launch_ssm_recurrent(p, static_cast<hipStream_t>(stream)));
    p.seg = plan.seg;
    p.map = plan.map;
    if (plan.map.slabs > 0) {
        p.slabs = static_cast<float *>(a.workspace);
        p.logs = p.slabs + plan.map.slabs * plan.slab;
    }
    return launched(kda::layer::launch_ssm_chunk(p, static_cast<hipStream_t>(stream)));
}

namespace {

// Sizes of a delta rule call: KDA_OK and the sequences, or what is wrong.
kda_status check_delta_sizes(const kda_delta_args &a, Seqs *s)
{
    if ((a.K != 64 && a.K != 128 && a.K != 256) || a.V < 16 || a.V > kDeltaMaxV || a.V % 16 != 0 || a.seg_tokens < 0 ||
        a.seg_tokens % kDeltaTile != 0)
        return KDA_ERR_SHAPE;
    if (a.H < 1 || a.H > 65536 || a.T > kDeltaMaxTokens)
        return KDA_ERR_SIZE;
    if (a.G < 1 || a.H % a.G != 0)
        return KDA_ERR_SHAPE;
    const kda_status st = check_seqs(a.cu_seqlens, a.num_seqs, a.B, a.T, s);
    int64_t rows, n;
    if (st == KDA_OK && (!mul_ok(a.B, a.T, &rows) || !mul_ok(rows, a.H * a.V * 2, &n) ||
                         !mul_ok(s->N, a.H * a.K * a.V * 4, &n) || s->N * a.H > INT32_MAX))
        return KDA_ERR_SIZE;
    return st;
}

// How a delta rule call with valid sizes runs.
struct DeltaPlan {
    bool recurrent = false;
    int64_t seg = 0;  // tokens a segment (chunked kernel), 0: whole sequences
    kda::layer::SlabMap map = {};
    int64_t bytes = 0;  // workspace
};

// The token recurrence, against the chunked kernel, in us for 32 heads of 128 and fp32 states:
// - up to kDeltaRecurrentMaxTokens tokens a sequence.  64 sequences of 1 / 4 / 8 / 12 / 16
//   tokens 45 / 56 / 82 / 110 / 137 (chunked 113 / 111 / 114 / 114 / 117), 8 of them
//   12 / 12 / 15 / 19 / 24 (15 / 15 / 16 / 16 / 16).
// - packed sequences, whose lengths the host does not know, of up to two tokens
//   on average: 64 of 1 / 2 tokens 44 / 47 (133 / 134), one of 33 and 31 of 1 38 (66), one of
//   64 and 63 of none 68 (75), 256 of 1 and one of 257 309 (470); but where nearly all are empty
//   one long sequence is gone through alone: 2048 tokens and 1023 of none 1933 (841).
// Of the others, few chains are cut into segments: as many as leave no compute unit of
// 256 a second workgroup in the pass over own states, which has V + K columns, 128 a
// workgroup, and of eight tiles at least.  That pass does again what the output
// pass does, so a sequence has to be 2.5 segments long, or packed ones of unequal lengths 1.9 on
// average, since the longest of these is what segments shorten.  At 1.9 to 2 segments both take
// about as long (-2 to +6 % by the mean); at 2.5 cutting wins.  In us, whole and cut, heads of 128 (packed ones: five sets of
// lengths and their mean):
//   one sequence of 8191 tokens, 12 heads of 64 x 96   391  107 (10 segments)
//   one of 8192, 32 / 40 / 64 heads                    450  320 (4) / 464  379 (3) / 468  545 (2)
//   one of 1024, 32 heads                              61   70 (2)
//   16384 tokens in 2 packed, 24 heads                 536 to 808, 662  551 to 562, 556 (5 in all, 2.5 each)
//   in 4, 12 heads                                     298 to 520, 375  294 to 407, 322 (10, 2.5)
//   in 8, 6 heads                                      182 to 246, 207  164 to 226, 179 (21, 2.5)
//   in 8, 8 heads                                      183 to 247, 207  194 to 264, 210 (16, 2.0)
//   in 10, 6 heads                                     155 to 179, 165  163 to 221, 175 (21, 2.0)
//   in 6, 10 heads                                     206 to 344, 257  249 to 254, 252 (12, 1.9)
//   in 9, 7 heads                                      166 to 205, 185  181 to 249, 197 (18, 1.9)
//   in 8, 16 heads                                     194 to 258, 219  345 (8, 1.0)
//   8000 in 12, 4 heads                                72 to 77, 74     87 to 90, 88 (16, 1.3)
// Packed calls of more sequences than that many segments stay whole, also where one is far
// longer than the others, which the host does not know: a prompt of 16384 tokens and 15 / 63 /
// 255 single ones, 32 heads 1460 / 1462 / 1464, in segments of 4096 699 / 709 / 1032.
// False if the workspace overflows.
bool delta_plan(const kda_delta_args &a, const Seqs &s, DeltaPlan *plan)
{
    constexpr int64_t kTarget = 256, kColumns = 128, kShortest = 8 * kDeltaTile;
    if (s.T <= (s.cu ? 2 * s.N : kDeltaRecurrentMaxTokens) && (a.seg_tokens == 0 || a.seg_tokens >= s.T)) {
        plan->recurrent = true;
        return true;
    }
    int64_t seg = a.seg_tokens;
    if (seg == 0) {
        const int64_t parts = kTarget / (a.H * ((a.V + a.K + kColumns - 1) / kColumns));  // segments in all
        if (s.N < 1 || parts < s.N)
            return true;
        const bool unequal = s.cu && s.N > 1;
        const int64_t all = unequal ? parts : parts / s.N, each = unequal ? s.T / s.N : s.T;
        seg = std::max(((s.T + all - 1) / all + kDeltaTile - 1) / kDeltaTile * kDeltaTile, kShortest);
        if (8 * each < (unequal ? 15 : 20) * seg)
            return true;
    }
    if (seg >= s.T)
        return true;
    plan->seg = seg;
    plan->map = kda::layer::slab_map(s, seg);
    int64_t n;
    return mul_ok(a.H * (a.V + a.K), a.K * 4, &n) && mul_ok(plan->map.slabs, n, &plan->bytes);
}

}  // namespace

extern "C" int64_t kda_delta_workspace_bytes(const kda_delta_args *args)
{
    Seqs s;
    DeltaPlan plan;
    if (!args || check_delta_sizes(*args, &s) != KDA_OK || !delta_plan(*args, s, &plan))
        return -1;
    return plan.bytes;
}

extern "C" kda_status kda_delta_fwd(const kda_delta_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_delta_args &a = *args;
    if (a.reserved != 0)
        return KDA_ERR_OPTION;
    DeltaParams p = {};
    kda_status st = check_delta_sizes(a, &p.seqs);
    if (st == KDA_OK && (!std::isfinite(a.scale) || !fp32_scale(a.scale)))
        st = KDA_ERR_SCALE;
    if (st == KDA_OK)
        st = check_states(a.initial_state, a.initial_state_dtype, a.final_state, a.final_state_dtype);
    if (st != KDA_OK)
        return st;
    DeltaPlan plan;
    if (!delta_plan(a, p.seqs, &plan))
        return KDA_ERR_SIZE;
    const int64_t tokens = a.B * a.T;
    const int64_t state = p.seqs.N * a.H * a.K * a.V;
    int64_t nq, nk, nv, ng, nb;
    if (!extent(a.B, a.q_stride_b, a.T, a.q_stride_t, a.G * a.K, 2, &nq) ||
        !extent(a.B, a.k_stride_b, a.T, a.k_stride_t, a.G * a.K, 2, &nk) ||
        !extent(a.B, a.v_stride_b, a.T, a.v_stride_t, a.H * a.V, 2, &nv) ||
        !extent(a.B, a.g_stride_b, a.T, a.g_stride_t, a.H, 2, &ng) ||
        !extent(a.B, a.beta_stride_b, a.T, a.beta_stride_t, a.H, 2, &nb))
        return KDA_ERR_STRIDE;
    if ((p.seqs.cu ? a.T > 1 : a.T > kDeltaRecurrentMaxTokens) &&  // one rule of sizes, whichever kernel runs
        (a.q_stride_t > kDeltaMaxStride || a.k_stride_t > kDeltaMaxStride || a.v_stride_t > kDeltaMaxStride ||
         a.g_stride_t > kDeltaMaxStride || a.beta_stride_t > kDeltaMaxStride))
        return KDA_ERR_STRIDE;
    if ((tokens > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.out)) || !a.A_log)
        return KDA_ERR_NULL_POINTER;
    const Span sq = span(a.q, nq), sk = span(a.k, nk), sv = span(a.v, nv), sg = span(a.g, ng), sb = span(a.beta, nb),
               sA = span(a.A_log, a.H * 4), sd = span(a.dt_bias, a.H * 4),
               su = span(a.cu_seqlens, a.cu_seqlens ? (p.seqs.N + 1) * 8 : 0), so = span(a.out, tokens * a.H * a.V * 2),
               si = span(a.initial_state, a.initial_state ? state * bytes_of(a.initial_state_dtype) : 0),
               sf = span(a.final_state, a.final_state ? state * bytes_of(a.final_state_dtype) : 0);
    if (any_overlap(so, {sq, sk, sv, sg, sb, sA, sd, su, si, sf}) ||
        any_overlap(sf, {sq, sk, sv, sg, sb, sA, sd, su}) || (sf.overlaps(si) && a.final_state != a.initial_state))
        return KDA_ERR_ALIAS;
    if (misaligned(a.q, 2) || misaligned(a.k, 2) || misaligned(a.v, 2) || misaligned(a.g, 2) || misaligned(a.beta, 2) ||
        misaligned(a.out, 16) || misaligned(a.initial_state, 16) || misaligned(a.final_state, 16) ||
        misaligned(a.A_log, 4) || misaligned(a.dt_bias, 4) || misaligned(a.cu_seqlens, 8))
        return KDA_ERR_ALIGNMENT;
    if (plan.bytes > 0 && (!a.workspace || a.workspace_bytes < plan.bytes || misaligned(a.workspace, 16) ||
                           any_overlap(span(a.workspace, plan.bytes), {sq, sk, sv, sg, sb, sA, sd, su, so, si, sf})))
        return KDA_ERR_WORKSPACE;
    if (p.seqs.N == 0 || (tokens == 0 && !a.final_state))
        return KDA_OK;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint16_t *>(a.k);
    p.v = static_cast<const uint16_t *>(a.v);
    p.g = static_cast<const uint16_t *>(a.g);
    p.beta = static_cast<const uint16_t *>(a.beta);
    p.out = static_cast<uint16_t *>(a.out);
    p.qb = a.q_stride_b;
    p.qt = a.q_stride_t;
    p.kb = a.k_stride_b;
    p.kt = a.k_stride_t;
    p.vb = a.v_stride_b;
    p.vt = a.v_stride_t;
    p.gb = a.g_stride_b;
    p.gt = a.g_stride_t;
    p.bb = a.beta_stride_b;
    p.bt = a.beta_stride_t;
    p.A_log = a.A_log;
    p.dt_bias = a.dt_bias;
    p.init_state = a.initial_state;
    p.final_state = a.final_state;
    p.init_kind = a.initial_state ? a.initial_state_dtype : KDA_DTYPE_NONE;
    p.final_kind = a.final_state ? a.final_state_dtype : KDA_DTYPE_NONE;
    p.H = a.H;
    p.G = a.G;
    p.K = a.K;
    p.V = a.V;
    p.scale = static_cast<float>(a.scale);
    p.seg = plan.seg;
    p.map = plan.map;
    p.slabs = static_cast<float *>(a.workspace);
    return launched((plan.recurrent ? launch_delta_recurrent : launch_delta_chunk)(p, static_cast<hipStream_t>(stream)));
}

extern "C" kda_status kda_gated_norm(const kda_gated_norm_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_gated_norm_args &a = *args;
    if (a.reserved != 0 || !flag(a.gate_first) ||
        (a.gate && a.activation != KDA_ACT_SIGMOID && a.activation != KDA_ACT_SILU))
        return KDA_ERR_OPTION;
    if (a.D < 1 || a.D > kMaxChannels || a.group < 1 || a.group > kda::layer::kMaxNormSize || a.D % a.group != 0)
        return KDA_ERR_SHAPE;
    if (!valid_eps(a.eps))
        return KDA_ERR_SCALE;
    if (!bf16_or_fp32(a.weight_dtype))
        return KDA_ERR_DTYPE;
    int64_t out_bytes, nx, ng;
    if (a.rows < 0 || !mul_ok(a.rows, 2 * a.D, &out_bytes))
        return KDA_ERR_SIZE;
    if (!extent(1, 0, a.rows, a.x_stride, a.D, 2, &nx) || !extent(1, 0, a.rows, a.gate_stride, a.D, 2, &ng))
        return KDA_ERR_STRIDE;
    if (!a.weight || (a.rows > 0 && (!a.x || !a.out)))
        return KDA_ERR_NULL_POINTER;
    const int64_t we = bytes_of(a.weight_dtype);
    if (any_overlap(span(a.out, out_bytes), {span(a.x, nx), span(a.gate, ng), span(a.weight, a.D * we)}))
        return KDA_ERR_ALIAS;
    if (misaligned(a.x, 2) || misaligned(a.gate, 2) || misaligned(a.weight, we) || misaligned(a.out, 16))
        return KDA_ERR_ALIGNMENT;
    if (a.rows == 0)
        return KDA_OK;
    kda::layer::GatedParams p = {};
    p.x = static_cast<const uint16_t *>(a.x);
    p.gate = static_cast<const uint16_t *>(a.gate);
    p.xr = a.x_stride;
    p.gr = a.gate_stride;
    p.weight = a.weight;
    p.weight_kind = a.weight_dtype;
    p.out = static_cast<uint16_t *>(a.out);
    p.rows = a.rows;
    p.D = a.D;
    p.group = a.group;
    p.act = a.activation;
    p.gate_first = a.gate_first;
    p.eps = kda::layer::norm_eps(a.eps);
    return launched(kda::layer::launch_gated_norm(p, static_cast<hipStream_t>(stream)));
}

extern "C" kda_status kda_residual_norm(const kda_residual_norm_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_residual_norm_args &a = *args;
    if (a.reserved != 0)
        return KDA_ERR_OPTION;
    if (a.D < 1 || a.D > kda::layer::kMaxNormSize)
        return KDA_ERR_SHAPE;
    if (!valid_eps(a.eps) || !fp32_scale(a.residual_scale) || !fp32_scale(a.block_scale))
        return KDA_ERR_SCALE;
    if ((a.residual && !bf16_or_fp32(a.residual_dtype)) || (a.residual_out && !bf16_or_fp32(a.residual_out_dtype)) ||
        (a.post_weight && !bf16_or_fp32(a.post_weight_dtype)) || (a.gate && !bf16_or_fp32(a.gate_dtype)) ||
        (a.weight && !bf16_or_fp32(a.weight_dtype)))
        return KDA_ERR_DTYPE;
    int64_t cells, nx, ng = 0;
    if (a.rows < 0 || !mul_ok(a.rows, 4 * a.D, &cells) || (a.gate && a.gate_period < 1))
        return KDA_ERR_SIZE;
    cells /= 4;
    if (!extent(1, 0, a.rows, a.x_stride, a.D, 2, &nx) ||
        (a.gate && !extent(1, 0, a.rows > 0 ? (a.rows - 1) / a.gate_period + 1 : 0, a.gate_stride, a.D,
                           bytes_of(a.gate_dtype), &ng)))
        return KDA_ERR_STRIDE;
    if ((a.rows > 0 && (!a.x || (!a.out && !a.residual_out))) || (a.out && !a.weight) || (a.weight && !a.out && a.rows > 0))
        return KDA_ERR_NULL_POINTER;
    const Span sx = span(a.x, nx), sr = span(a.residual, a.residual ? cells * bytes_of(a.residual_dtype) : 0),
               sq = span(a.residual_out, a.residual_out ? cells * bytes_of(a.residual_out_dtype) : 0),
               sp = span(a.post_weight, a.post_weight ? a.D * bytes_of(a.post_weight_dtype) : 0), sg = span(a.gate, ng),
               sw = span(a.weight, a.weight ? a.D * bytes_of(a.weight_dtype) : 0), so = span(a.out, cells * 2);
    const bool in_place = a.residual_out == a.residual && a.residual_out_dtype == a.residual_dtype;
    if (any_overlap(so, {sx, sr, sq, sp, sg, sw}) || any_overlap(sq, {sx, sp, sg, sw}) ||
        (sq.overlaps(sr) && !in_place))
        return KDA_ERR_ALIAS;
    if (misaligned(a.x, 2) || misaligned(a.out, 16) || misaligned(a.residual, a.residual ? bytes_of(a.residual_dtype) : 1) ||
        misaligned(a.residual_out, a.residual_out ? 16 : 1) ||
        misaligned(a.post_weight, a.post_weight ? bytes_of(a.post_weight_dtype) : 1) ||
        misaligned(a.gate, a.gate ? bytes_of(a.gate_dtype) : 1) ||
        misaligned(a.weight, a.weight ? bytes_of(a.weight_dtype) : 1))
        return KDA_ERR_ALIGNMENT;
    if (a.rows == 0)
        return KDA_OK;
    kda::layer::ResidParams p = {};
    p.x = static_cast<const uint16_t *>(a.x);
    p.xr = a.x_stride;
    p.residual = a.residual;
    p.residual_out = a.residual_out;
    p.residual_kind = a.residual_dtype;
    p.residual_out_kind = a.residual_out_dtype;
    p.post_weight = a.post_weight;
    p.post_kind = a.post_weight_dtype;
    p.weight = a.weight;
    p.weight_kind = a.weight_dtype;
    p.gate = a.gate;
    p.gate_kind = a.gate_dtype;
    p.gr = a.gate_stride;
    p.gate_period = a.gate_period;
    p.out = static_cast<uint16_t *>(a.out);
    p.rows = a.rows;
    p.D = a.D;
    p.residual_scale = static_cast<float>(a.residual_scale);
    p.block_scale = static_cast<float>(a.block_scale);
    p.eps = kda::layer::norm_eps(a.eps);
    return launched(kda::layer::launch_residual_norm(p, static_cast<hipStream_t>(stream)));
}
