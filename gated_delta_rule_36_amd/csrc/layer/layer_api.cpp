// C-ABI front end of the layer operators: argument checks on the host, then
// the hand-off to the kernels.  Nothing here touches device memory.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kda.h"
#include "layer_internal.h"

namespace {

using kda::layer::Seqs;

constexpr int64_t kMaxChannels = int64_t(1) << 24;

bool mul_ok(int64_t a, int64_t b, int64_t *r) { return !__builtin_mul_overflow(a, b, r); }
bool add_ok(int64_t a, int64_t b, int64_t *r) { return !__builtin_add_overflow(a, b, r); }

bool bf16_or_fp32(int32_t d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32; }
int64_t bytes_of(int32_t d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }
bool flag(int32_t v) { return v == 0 || v == 1; }
bool valid_eps(double e) { return std::isfinite(e) && e >= 0.0; }
// The kernels multiply in fp32: a scale has to be 0 or normal there.
bool fp32_scale(double s) { return s == 0.0 || std::isnormal(static_cast<float>(s)); }

// Byte range of a buffer.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool overlaps(const Span &o) const { return lo < o.hi && o.lo < hi; }
};
Span span(const void *p, int64_t bytes)
{
    Span s;
    if (p && bytes > 0) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + static_cast<uintptr_t>(bytes);
    }
    return s;
}
bool any_overlap(const Span &out, std::initializer_list<Span> inputs)
{
    for (const Span &s : inputs)
        if (out.overlaps(s))
            return true;
    return false;
}

bool misaligned(const void *p, uintptr_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a != 0; }

// Bytes from the first to past the last element of `outer` x `inner` rows of
// `width` adjacent elements with the given strides; false on a negative
// stride or overflow.
bool extent(int64_t outer, int64_t stride_o, int64_t inner, int64_t stride_i, int64_t width, int64_t elem,
            int64_t *bytes)
{
    int64_t a = 0, b = 0, n = 0;
    if (stride_o < 0 || stride_i < 0)
        return false;
    if (outer == 0 || inner == 0 || width == 0) {
        *bytes = 0;
        return true;
    }
    return mul_ok(outer - 1, stride_o, &a) && mul_ok(inner - 1, stride_i, &b) && add_ok(a, b, &n) &&
           add_ok(n, width, &n) && mul_ok(n, elem, bytes);
}

// The batch of sequences a call names: KDA_OK, or what is wrong with it.
kda_status check_seqs(const int64_t *cu, int64_t num_seqs, int64_t B, int64_t T, Seqs *s)
{
    if (B < 1 || T < 0 || T > INT32_MAX)
        return KDA_ERR_SIZE;
    if (cu && (B != 1 || num_seqs < 0))
        return KDA_ERR_VARLEN_BATCH;
    s->cu = cu;
    s->N = cu ? num_seqs : B;
    s->T = T;
    return s->N > INT32_MAX ? KDA_ERR_SIZE : KDA_OK;
}

kda_status check_states(const void *init, int32_t init_dtype, const void *fin, int32_t fin_dtype)
{
    if (init && !bf16_or_fp32(init_dtype))
        return init_dtype == KDA_DTYPE_NONE ? KDA_ERR_NULL_POINTER : KDA_ERR_STATE_DTYPE;
    if (fin && !bf16_or_fp32(fin_dtype))
        return fin_dtype == KDA_DTYPE_NONE ? KDA_ERR_NULL_POINTER : KDA_ERR_STATE_DTYPE;
    return init && fin && init_dtype != fin_dtype ? KDA_ERR_STATE_DTYPE : KDA_OK;
}

kda_status launched(hipError_t e)
{
    return e == hipSuccess ? KDA_OK : e == hipErrorInvalidConfiguration ? KDA_ERR_SIZE : KDA_ERR_LAUNCH;
}

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
