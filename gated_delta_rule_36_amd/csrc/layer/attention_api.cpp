// C-ABI front end of the attention layers' operators: argument checks on the
// host, then the hand-off to the kernels.  Nothing here touches device memory.
#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "layer_checks.h"

namespace {

using namespace kda::layer;

// Bytes from the first to past the last element of a cache of adjacent
// channels; false on a negative stride or overflow.
bool cache_extent(int64_t pages, int64_t page_size, int64_t heads, int64_t D, const CacheStrides &s, int64_t *bytes)
{
    int64_t a, b, c, n;
    if (s.page < 0 || s.token < 0 || s.head < 0)
        return false;
    if (pages == 0) {
        *bytes = 0;
        return true;
    }
    return mul_ok(pages - 1, s.page, &a) && mul_ok(page_size - 1, s.token, &b) && mul_ok(heads - 1, s.head, &c) &&
           add_ok(a, b, &n) && add_ok(n, c, &n) && add_ok(n, D, &n) && mul_ok(n, 2, bytes);
}

// Whether no two rows of `width` elements share memory, given their dimensions
// as (stride, size): from the smallest stride up, each step passes all that lies
// below it.
template <size_t N>
bool rows_apart(int64_t width, std::pair<int64_t, int64_t> (&&dims)[N])
{
    std::sort(dims, dims + N);
    int64_t below = width;
    for (const auto &d : dims) {
        if (d.second <= 1)
            continue;
        if (d.first < below)
            return false;
        below += (d.second - 1) * d.first;
    }
    return true;
}
bool places_apart(int64_t pages, int64_t page_size, int64_t heads, int64_t D, const CacheStrides &s)
{
    return rows_apart(D, {{s.page, pages}, {s.token, page_size}, {s.head, heads}});
}

// Widths, weights and scales of the rotation's two entry points.
kda_status check_rotation(int64_t D, int64_t R, bool rotates, const void *weight, int32_t weight_dtype, const void *weight2,
                          int32_t weight2_dtype, double eps, double scale)
{
    if (D < 2 || D > kMaxHeadChannels || D % 2 != 0 || (rotates && (R < 2 || R > D || R % 2 != 0)))
        return KDA_ERR_SHAPE;
    if (!valid_eps(eps) || !std::isfinite(scale) || !fp32_scale(scale))
        return KDA_ERR_SCALE;
    if ((weight && !bf16_or_fp32(weight_dtype)) || (weight2 && !bf16_or_fp32(weight2_dtype)))
        return KDA_ERR_DTYPE;
    return KDA_OK;
}

// Tokens of a call: KDA_OK, or a size that is refused.
kda_status check_tokens(int64_t B, int64_t T, int64_t heads, int64_t D, int64_t *tokens)
{
    int64_t n;
    if (B < 0 || T < 0 || T > INT32_MAX || heads < 0 || heads > 65536 || !mul_ok(B, T, tokens) ||
        !mul_ok(*tokens, 8, &n) || !mul_ok(*tokens, 2 * (heads > 0 ? heads : 1) * D, &n))
        return KDA_ERR_SIZE;
    return KDA_OK;
}

}  // namespace

extern "C" kda_status kda_qk_norm_rotary(const kda_rotary_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_rotary_args &a = *args;
    if (a.reserved != 0 || !flag(a.interleaved))
        return KDA_ERR_OPTION;
    kda_status st = check_rotation(a.D, a.R, a.positions != nullptr, a.q_weight, a.q_weight_dtype, a.k_weight,
                                   a.k_weight_dtype, a.eps, a.rotary_scale);
    int64_t tokens = 0;
    if (st == KDA_OK)
        st = a.Hq < 1 ? KDA_ERR_SIZE : check_tokens(a.B, a.T, a.Hq, a.D, &tokens);
    if (st == KDA_OK)
        st = check_tokens(a.B, a.T, a.Hk, a.D, &tokens);
    if (st != KDA_OK)
        return st;
    int64_t nq, nk;
    if (!extent(a.B, a.q_stride_b, a.T, a.q_stride_t, a.Hq * a.D, 2, &nq) ||
        !extent(a.B, a.k_stride_b, a.T, a.k_stride_t, a.Hk * a.D, 2, &nk))
        return KDA_ERR_STRIDE;
    if ((tokens > 0 && (!a.q || !a.q_out || (a.Hk > 0 && (!a.k || !a.k_out)))) || (a.positions && !a.inv_freq) ||
        (a.inv_freq && !a.positions && tokens > 0))
        return KDA_ERR_NULL_POINTER;
    const int64_t qo = tokens * a.Hq * a.D * 2, ko = tokens * a.Hk * a.D * 2;
    const Span sq = span(a.q, nq), sk = span(a.k, nk), soq = span(a.q_out, qo), sok = span(a.k_out, ko),
               sp = span(a.positions, a.positions ? tokens * 8 : 0), sf = span(a.inv_freq, a.positions ? a.R * 2 : 0),
               sw = span(a.q_weight, a.q_weight ? a.D * bytes_of(a.q_weight_dtype) : 0),
               su = span(a.k_weight, a.k_weight ? a.D * bytes_of(a.k_weight_dtype) : 0);
    // in place: the input is contiguous, too (strides of single rows do not count)
    const auto in_place = [&](const void *x, const void *out, int64_t sb, int64_t st_, int64_t row) {
        return x == out && (a.T <= 1 || st_ == row) && (a.B <= 1 || sb == a.T * row);
    };
    if (any_overlap(soq, {sk, sok, sp, sf, sw, su}) || any_overlap(sok, {sq, sp, sf, sw, su}) ||
        (soq.overlaps(sq) && !in_place(a.q, a.q_out, a.q_stride_b, a.q_stride_t, a.Hq * a.D)) ||
        (sok.overlaps(sk) && !in_place(a.k, a.k_out, a.k_stride_b, a.k_stride_t, a.Hk * a.D)))
        return KDA_ERR_ALIAS;
    if (misaligned(a.q, 2) || misaligned(a.k, 2) || misaligned(a.q_out, 16) || misaligned(a.k_out, 16) ||
        misaligned(a.positions, 8) || misaligned(a.inv_freq, 4) ||
        misaligned(a.q_weight, a.q_weight ? bytes_of(a.q_weight_dtype) : 1) ||
        misaligned(a.k_weight, a.k_weight ? bytes_of(a.k_weight_dtype) : 1))
        return KDA_ERR_ALIGNMENT;
    if (tokens == 0)
        return KDA_OK;
    RotaryParams p = {};
    p.x = static_cast<const uint16_t *>(a.q);
    p.y = static_cast<const uint16_t *>(a.k);
    p.xb = a.q_stride_b;
    p.xt = a.q_stride_t;
    p.yb = a.k_stride_b;
    p.yt = a.k_stride_t;
    p.x_out = static_cast<uint16_t *>(a.q_out);
    p.y_out = static_cast<uint16_t *>(a.k_out);
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.x_weight = a.q_weight;
    p.y_weight = a.k_weight;
    p.x_kind = a.q_weight_dtype;
    p.y_kind = a.k_weight_dtype;
    p.B = a.B;
    p.T = a.T;
    p.first = static_cast<int>(a.Hq);
    p.second = static_cast<int>(a.Hk);
    p.D = static_cast<int>(a.D);
    p.R = static_cast<int>(a.R);
    p.interleaved = a.interleaved;
    p.eps = norm_eps(a.eps);
    p.scale = static_cast<float>(a.rotary_scale);
    return launched(launch_rotary(p, static_cast<hipStream_t>(stream)));
}

extern "C" kda_status kda_append_kv(const kda_append_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_append_args &a = *args;
    if (a.reserved != 0 || !flag(a.interleaved))
        return KDA_ERR_OPTION;
    kda_status st = check_rotation(a.D, a.R, a.positions != nullptr, a.weight, a.weight_dtype, nullptr, 0, a.eps, a.rotary_scale);
    int64_t tokens = 0, slots, n;
    if (st == KDA_OK)
        st = a.Hk < 1 ? KDA_ERR_SIZE : check_tokens(a.B, a.T, a.Hk, a.D, &tokens);
    if (st != KDA_OK)
        return st;
    if (a.pages < 0 || a.page_size < 1 || !mul_ok(a.pages, a.page_size, &slots) || !mul_ok(slots, 2 * a.Hk * a.D, &n))
        return KDA_ERR_SIZE;
    const CacheStrides kc = {a.k_cache_stride_page, a.k_cache_stride_token, a.k_cache_stride_head},
                       vc = {a.v_cache_stride_page, a.v_cache_stride_token, a.v_cache_stride_head};
    int64_t nk, nv, nkc, nvc;
    if (!extent(a.B, a.k_stride_b, a.T, a.k_stride_t, a.Hk * a.D, 2, &nk) ||
        !extent(a.B, a.v_stride_b, a.T, a.v_stride_t, a.Hk * a.D, 2, &nv) ||
        !cache_extent(a.pages, a.page_size, a.Hk, a.D, kc, &nkc) ||
        !cache_extent(a.pages, a.page_size, a.Hk, a.D, vc, &nvc) || !places_apart(a.pages, a.page_size, a.Hk, a.D, kc) ||
        !places_apart(a.pages, a.page_size, a.Hk, a.D, vc))
        return KDA_ERR_STRIDE;
    if ((tokens > 0 && (!a.k || !a.v || !a.slots || (slots > 0 && (!a.k_cache || !a.v_cache)))) ||
        (a.positions && !a.inv_freq) || (a.inv_freq && !a.positions && tokens > 0))
        return KDA_ERR_NULL_POINTER;
    const Span sk = span(a.k, nk), sv = span(a.v, nv), skc = span(a.k_cache, nkc), svc = span(a.v_cache, nvc),
               ss = span(a.slots, tokens * 8), sp = span(a.positions, a.positions ? tokens * 8 : 0),
               sf = span(a.inv_freq, a.positions ? a.R * 2 : 0),
               sw = span(a.weight, a.weight ? a.D * bytes_of(a.weight_dtype) : 0);
    // The two caches may be interleaved in one buffer (a dimension of keys and
    // values): apart if every row of one lies in the gaps of the other.
    const auto woven = [&] {
        const int64_t gap = reinterpret_cast<intptr_t>(a.v_cache) - reinterpret_cast<intptr_t>(a.k_cache);
        if (gap % 2 != 0 || kc.page != vc.page || kc.token != vc.token || kc.head != vc.head)
            return false;
        // as a fourth dimension of size 2
        return rows_apart(a.D, {{kc.page, a.pages}, {kc.token, a.page_size}, {kc.head, a.Hk}, {(gap < 0 ? -gap : gap) / 2, 2}});
    };
    if (any_overlap(skc, {sk, sv, ss, sp, sf, sw}) || any_overlap(svc, {sk, sv, ss, sp, sf, sw}) ||
        (skc.overlaps(svc) && !woven()))
        return KDA_ERR_ALIAS;
    if (misaligned(a.k, 2) || misaligned(a.v, 2) || misaligned(a.k_cache, 2) || misaligned(a.v_cache, 2) ||
        misaligned(a.slots, 8) || misaligned(a.positions, 8) || misaligned(a.inv_freq, 4) ||
        misaligned(a.weight, a.weight ? bytes_of(a.weight_dtype) : 1))
        return KDA_ERR_ALIGNMENT;
    if (tokens == 0 || slots == 0)
        return KDA_OK;
    RotaryParams p = {};
    p.x = static_cast<const uint16_t *>(a.k);
    p.y = static_cast<const uint16_t *>(a.v);
    p.xb = a.k_stride_b;
    p.xt = a.k_stride_t;
    p.yb = a.v_stride_b;
    p.yt = a.v_stride_t;
    p.x_out = static_cast<uint16_t *>(a.k_cache);
    p.y_out = static_cast<uint16_t *>(a.v_cache);
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.x_weight = a.weight;
    p.x_kind = a.weight_dtype;
    p.B = a.B;
    p.T = a.T;
    p.first = p.second = static_cast<int>(a.Hk);
    p.D = static_cast<int>(a.D);
    p.R = static_cast<int>(a.R);
    p.interleaved = a.interleaved;
    p.eps = norm_eps(a.eps);
    p.scale = static_cast<float>(a.rotary_scale);
    p.slots = a.slots;
    p.slot_count = slots;
    p.page_size = a.page_size;
    p.xc = kc;
    p.yc = vc;
    return launched(launch_rotary(p, static_cast<hipStream_t>(stream)));
}

namespace {

kda_status check_attention_sizes(const kda_attention_args &a)
{
    if (a.D < 16 || a.D > kAttentionMaxD || a.D % 16 != 0 || a.Hk < 1 || a.Hq < 1 || a.Hq % a.Hk != 0)
        return KDA_ERR_SHAPE;
    int64_t n;
    if (a.N < 0 || a.N > INT32_MAX || a.Hq > 65536 || a.pages < 0 || a.pages > INT32_MAX || a.page_size < 1 ||
        a.page_size > INT32_MAX || a.table_width < 0 || a.window < 0 || !mul_ok(a.table_width, a.page_size, &n) ||
        n > INT32_MAX - 65536 || !mul_ok(a.N, a.Hq * a.D * 4, &n))
        return KDA_ERR_SIZE;
    return KDA_OK;
}

// How the tokens of a sequence are cut into splits, by sizes alone: a context is
// taken as long as its table allows, or its window, since the host does not know the
// lengths.  So a table much wider than the contexts leaves few waves for each: 64
// requests of 2000 tokens, 8 key heads, with a table for as many, 8 and 64 times as many
// 118 / 157 / 945 us; of 16384 812 / 1067 / 7611; 256 of 1024 217 / 1002 / 1953.
// Times in us, 128 channels; n x t are n sequences of t tokens in all, of lengths that differ.
// - At most kShared tokens: one split, shared by a workgroup's four waves, and
//   neither a workspace nor a second launch.
// - pairs (of a sequence and up to 16 query heads of a key head) times tokens
//   below kFew: kGroups splits over all, of one workgroup's four waves each, of
//   at most kSharedMost tokens.  A wave alone on as many: 1 x 131071 tokens, 2 key heads
//   40 (shared 37), 1 x 16384 19 (15), 4 x 65536 30 (26), 8 x 16384 of 4 key heads 21
//   (19).  Splits of 1024: 38, 26, 30, 27.
// - Above: one split a wave, whose neighbours take the other key heads of the
//   same tokens and so read whole rows of the cache between them.  16 x 32768, 8 key heads 42
//   (shared 44).  As many splits as make kTarget waves: 64 x 131072 tokens at the
//   most each, 8 key heads, for 8192 / 16384 / 32768 / 65536 waves 1034 / 886 / 826 / 857.
//   All splits have the same size, so that waves do the same work however lengths
//   differ; the same number of splits for every sequence took 991.
//   At least kFewest tokens, or up to kEnough if the splits still make kWaves: 16 x 32768, 8
//   key heads, splits of 128 / 160 / 192 / 320 tokens 42 / 46 / 51 / 55; 16 x 65536 68 / 70 / 65 / 81, 1 x
//   131072 129 / 118 / 118 / 118, 64 x 262144 of 4 key heads 136 / 134 / 131 / 137, 64 x 65536 of
//   8 with 256 channels 190 / 160 / 161 / 164.
constexpr int64_t kTarget = 32768, kFewest = 4 * kAttentionTile, kEnough = 6 * kAttentionTile, kWaves = 5120;
constexpr int64_t kShared = 1024, kSharedMost = 512, kGroups = 512, kFew = 327680;
int64_t longest(const kda_attention_args &a)
{
    const int64_t room = a.table_width * a.page_size;
    return a.window > 0 && a.window < room ? a.window : room;
}
int64_t attention_pairs(const kda_attention_args &a)
{
    // more than this no grid takes; times tokens it stays within 64 bits
    return std::min<int64_t>(a.N * a.Hk * ((a.Hq / a.Hk + kAttentionRows - 1) / kAttentionRows), INT32_MAX);
}
// Whether a workgroup's waves share a split.
bool attention_shared(const kda_attention_args &a)
{
    const int64_t most = longest(a);
    return most <= kShared || attention_pairs(a) * most < kFew;
}
int64_t attention_chunk(const kda_attention_args &a)
{
    const int64_t most = longest(a);
    if (most <= kShared)
        return kShared;
    if (attention_shared(a)) {
        constexpr int64_t kStep = 4 * kAttentionTile;
        const int64_t chunk = (attention_pairs(a) * most + kGroups - 1) / kGroups;
        return std::min(kSharedMost, (chunk + kStep - 1) / kStep * kStep);
    }
    const int64_t pairs = std::max(int64_t(1), attention_pairs(a)), parts = std::max(int64_t(1), kTarget / pairs);
    const int64_t least = std::min(kEnough, std::max(kFewest, pairs * most / kWaves));
    const int64_t chunk = std::max((most + parts - 1) / parts, least);
    return (chunk + kAttentionTile - 1) / kAttentionTile * kAttentionTile;
}
int64_t attention_splits(const kda_attention_args &a)
{
    const int64_t chunk = attention_chunk(a);
    return std::max(int64_t(1), (longest(a) + chunk - 1) / chunk);
}

int64_t attention_workspace(const kda_attention_args &a)
{
    const int64_t splits = attention_splits(a);
    return splits > 1 ? a.N * a.Hq * splits * (a.D + 2) * 4 : 0;
}

}  // namespace

extern "C" int64_t kda_paged_attention_workspace_bytes(const kda_attention_args *args)
{
    if (!args || check_attention_sizes(*args) != KDA_OK)
        return -1;
    return attention_workspace(*args);
}

extern "C" kda_status kda_paged_attention(const kda_attention_args *args, void *stream)
{
    if (!args)
        return KDA_ERR_NULL_POINTER;
    const kda_attention_args &a = *args;
    if (a.reserved != 0)
        return KDA_ERR_OPTION;
    const kda_status st = check_attention_sizes(a);
    if (st != KDA_OK)
        return st;
    if (!std::isfinite(a.scale) || !fp32_scale(a.scale))
        return KDA_ERR_SCALE;
    AttentionParams p = {};
    p.ks = {a.k_cache_stride_page, a.k_cache_stride_token, a.k_cache_stride_head};
    p.vs = {a.v_cache_stride_page, a.v_cache_stride_token, a.v_cache_stride_head};
    int64_t nq, nk, nv, nt;
    if (!extent(1, 0, a.N, a.q_stride, a.Hq * a.D, 2, &nq) || !extent(1, 0, a.N, a.table_stride, a.table_width, 4, &nt) ||
        !cache_extent(a.pages, a.page_size, a.Hk, a.D, p.ks, &nk) ||
        !cache_extent(a.pages, a.page_size, a.Hk, a.D, p.vs, &nv))
        return KDA_ERR_STRIDE;
    if (a.N > 0 && (!a.q || !a.out || !a.lengths || (a.table_width > 0 && !a.block_table) ||
                    (a.pages > 0 && (!a.k_cache || !a.v_cache))))
        return KDA_ERR_NULL_POINTER;
    const Span sq = span(a.q, nq), sk = span(a.k_cache, nk), sv = span(a.v_cache, nv), st_ = span(a.block_table, nt),
               sl = span(a.lengths, a.N * 4), so = span(a.out, a.N * a.Hq * a.D * 2),
               se = span(a.lse, a.lse ? a.N * a.Hq * 4 : 0);
    if (any_overlap(so, {sq, sk, sv, st_, sl, se}) || any_overlap(se, {sq, sk, sv, st_, sl}))
        return KDA_ERR_ALIAS;
    if (misaligned(a.q, 2) || misaligned(a.k_cache, 2) || misaligned(a.v_cache, 2) || misaligned(a.block_table, 4) ||
        misaligned(a.lengths, 4) || misaligned(a.out, 16) || misaligned(a.lse, 4))
        return KDA_ERR_ALIGNMENT;
    const int64_t bytes = attention_workspace(a);
    if (bytes > 0 && (!a.workspace || a.workspace_bytes < bytes || misaligned(a.workspace, 16) ||
                      any_overlap(span(a.workspace, bytes), {sq, sk, sv, st_, sl, so, se})))
        return KDA_ERR_WORKSPACE;
    if (a.N == 0)
        return KDA_OK;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint16_t *>(a.k_cache);
    p.v = static_cast<const uint16_t *>(a.v_cache);
    p.qr = a.q_stride;
    p.table = a.block_table;
    p.lengths = a.lengths;
    p.table_stride = a.table_stride;
    p.out = static_cast<uint16_t *>(a.out);
    p.lse = a.lse;
    p.N = a.N;
    p.Hq = a.Hq;
    p.Hk = a.Hk;
    p.D = a.D;
    p.pages = a.pages;
    p.width = a.table_width;
    p.window = a.window;
    p.page_size = static_cast<uint32_t>(a.page_size);
    // t / d for t < 2^31: with 2^s < d <= 2^(s+1) and m = ceil(2^(32+s) / d) < 2^32, m t / 2^(32+s) exceeds t / d by
    // less than t / 2^(32+s) < 2^-1-s, less than 1 / d, the least that a quotient below the next whole one lacks
    if (p.page_size > 1) {
        while ((int64_t(2) << p.page_shift) < a.page_size) ++p.page_shift;
        p.page_mul = static_cast<uint32_t>(((uint64_t(1) << (32 + p.page_shift)) + p.page_size - 1) / p.page_size);
    }
    p.splits = attention_splits(a);
    p.chunk = static_cast<int>(attention_chunk(a));
    p.shared = attention_shared(a);
    p.scale = static_cast<float>(a.scale);
    if (p.splits > 1) {
        p.part = static_cast<float *>(a.workspace);
        p.stats = p.part + a.N * a.Hq * p.splits * a.D;
    }
    return launched(launch_paged_attention(p, static_cast<hipStream_t>(stream)));
}
