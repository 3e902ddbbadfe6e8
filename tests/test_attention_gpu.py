"""qk_norm_rotary, append_kv and paged_attention on the GPU against their plain
64-bit forms: widths, pairings, strides, page sizes, lengths, masks."""
import math

import pytest
import torch

import gated_delta_rule_36_amd as kda
import mixer_ref as ref
from mixer_ref import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN = float("nan")


def rand(*shape, seed=0, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def freqs(R, base=10000.0):
    return base ** (-torch.arange(0, R, 2, dtype=torch.float32) / R)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ---------------------------------------------------------------------------
# qk_norm_rotary
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [
    (1, 1, 1, 1, 2, 2), (2, 3, 4, 2, 64, 64), (3, 1, 32, 4, 128, 128), (1, 70, 5, 1, 128, 32), (2, 5, 3, 0, 80, 20),
    (1, 9, 2, 2, 80, 80), (1, 4, 7, 3, 96, 24), (2, 2, 2, 1, 192, 64), (1, 3, 4, 4, 256, 256), (1, 2, 3, 1, 512, 512),
    (1, 5, 2, 1, 6, 4), (1, 5, 2, 1, 130, 66), (1, 3, 1, 1, 258, 258), (1, 3, 2, 1, 510, 2), (1, 3, 2, 2, 300, 100),
    (1, 3, 40, 40, 64, 64),
])
def test_rotary_shapes(B, T, Hq, Hk, D, R, interleaved):
    wide = rand(B, T, Hq + Hk + 1, D, seed=D + R)  # slices of a fused projection that starts at an odd place
    q, k = wide[:, :, 1:1 + Hq], wide[:, :, 1 + Hq:] if Hk else None
    pos = torch.randint(0, 5000, (B, T), generator=torch.Generator().manual_seed(1))
    qw, kw = rand(D, seed=2), rand(D, seed=3, dtype=torch.float32)
    f = freqs(R)
    gw = wide.cuda()
    qo = torch.full((B, T, Hq, D), NAN, dtype=BF, device="cuda")
    ko = torch.full((B, T, Hk, D), NAN, dtype=BF, device="cuda") if Hk else None
    kda.qk_norm_rotary(gw[:, :, 1:1 + Hq], gw[:, :, 1 + Hq:] if Hk else None, pos.cuda(), f.cuda(), qo, ko, qw.cuda(),
                       kw.cuda(), interleaved=interleaved, rotary_scale=1.25)
    check("q", qo, *ref.rotary(q, pos, f, qw, interleaved=interleaved, scale=1.25))
    if Hk:
        check("k", ko, *ref.rotary(k, pos, f, kw, interleaved=interleaved, scale=1.25))


def test_rotary_far_positions():
    """Positions up to 2^31: the fraction of a turn is that of the 64-bit product."""
    pos = torch.tensor([[0, 1, 131071, 1048577, 123456789, (1 << 31) - 1, -1, -1000003]])
    q = rand(1, 8, 2, 64, seed=5)
    f = freqs(64, 5e6)
    out = torch.empty(1, 8, 2, 64, dtype=BF, device="cuda")
    kda.qk_norm_rotary(q.cuda(), None, pos.cuda(), f.cuda(), out)
    check("q", out, *ref.rotary(q, pos, f))


def test_rotary_without_norm_is_exact_at_position_zero_and_without_positions_a_norm():
    q = rand(2, 3, 4, 64, seed=6)
    out = torch.empty(2, 3, 4, 64, dtype=BF, device="cuda")
    kda.qk_norm_rotary(q.cuda(), None, torch.zeros(2, 3, dtype=torch.int64, device="cuda"), freqs(64).cuda(), out)
    assert torch.equal(out.cpu(), q)
    w = rand(64, seed=7)
    kda.qk_norm_rotary(q.cuda(), None, None, None, out, None, w.cuda())
    check("norm", out, *ref.rotary(q, None, None, w))


@pytest.mark.parametrize("size", [1e-30, 1e-20, 1e20, 3e38, 0.0])
def test_rotary_norm_of_rows_beyond_fp32_squares(size):
    q = (rand(1, 2, 3, 96, seed=8, dtype=torch.float32).clamp(-1, 1) * size).to(BF)
    w = rand(96, seed=9)
    out = torch.empty(1, 2, 3, 96, dtype=BF, device="cuda")
    kda.qk_norm_rotary(q.cuda(), None, None, None, out, None, w.cuda(), eps=0.0 if size else 1e-6)
    check("q", out, *ref.rotary(q, None, None, w, eps=0.0 if size else 1e-6))


def test_rotary_non_finite_stays_in_its_head():
    q = rand(1, 4, 4, 64, seed=10)
    q[0, 1, 2, 5], q[0, 3, 0, 0] = math.inf, NAN
    out = torch.empty(1, 4, 4, 64, dtype=BF, device="cuda")
    w = rand(64, seed=11)
    kda.qk_norm_rotary(q.cuda(), None, torch.arange(4, device="cuda")[None].contiguous(), freqs(64).cuda(), out, None, w.cuda())
    clean = torch.ones(4, 4, dtype=torch.bool)
    clean[1, 2] = clean[3, 0] = False
    want, bound = ref.rotary(q, torch.arange(4)[None], freqs(64), w)
    check("q", out[0][clean.cuda()], want[0][clean], bound[0][clean])


def test_rotary_in_place():
    q, k = rand(2, 5, 4, 64, seed=12), rand(2, 5, 2, 64, seed=13)
    pos = torch.arange(10).view(2, 5)
    gq, gk = cuda(q, k)
    kda.qk_norm_rotary(gq, gk, pos.cuda(), freqs(64).cuda(), gq, gk)
    check("q", gq, *ref.rotary(q, pos, freqs(64)))
    check("k", gk, *ref.rotary(k, pos, freqs(64)))


# ---------------------------------------------------------------------------
# append_kv
# ---------------------------------------------------------------------------

def caches(layout, pages, size, H, D, seed):
    """Two caches filled with noise: pages of tokens, pages of heads, or both woven into one buffer."""
    if layout == "tokens":
        return rand(pages, size, H, D, seed=seed).cuda(), rand(pages, size, H, D, seed=seed + 1).cuda()
    if layout == "heads":
        return tuple(rand(pages, H, size, D, seed=seed + i).cuda().transpose(1, 2) for i in (0, 1))
    both = rand(pages, 2, size, H, D, seed=seed).cuda()
    return both[:, 0], both[:, 1]


@pytest.mark.parametrize("layout", ["tokens", "heads", "woven"])
@pytest.mark.parametrize("B,T,H,D,R,page", [
    (3, 1, 2, 128, 128, 16), (1, 37, 1, 64, 64, 16), (2, 9, 3, 80, 20, 1), (1, 20, 8, 128, 32, 7), (2, 4, 2, 18, 6, 5),
    (1, 3, 2, 256, 256, 64),
])
def test_append(layout, B, T, H, D, R, page):
    pages = 2 + 2 * B * T // page
    kv = rand(B, T, 2 * H, D, seed=20)
    k, v = kv[:, :, :H], kv[:, :, H:]
    gen = torch.Generator().manual_seed(21)
    slots = torch.randperm(pages * page, generator=gen)[:B * T].view(B, T)
    slots[0, 0] = -1
    if T > 2:
        slots[0, 2] = pages * page  # behind the cache
    pos = torch.randint(0, 100000, (B, T), generator=gen)
    w, f = rand(D, seed=22), freqs(R)
    kc, vc = caches(layout, pages, page, H, D, 23)
    want = ref.append(k, v, kc.cpu(), vc.cpu(), slots, pos, f, w)
    g = kv.cuda()
    kda.append_kv(g[:, :, :H], g[:, :, H:], kc, vc, slots.cuda(), pos.cuda(), f.cuda(), w.cuda())
    untouched = want[2] == 0
    assert torch.equal(kc.cpu().double()[untouched], want[0][untouched])
    check("k_cache", kc[(~untouched).cuda()], want[0][~untouched], want[2][~untouched])
    assert torch.equal(vc.cpu().double(), want[1])


def test_append_as_it_is_and_non_finite_values():
    """Without norm and rotation both are copies, bit for bit, NaN and infinities among them."""
    k, v = rand(1, 6, 2, 64, seed=30), rand(1, 6, 2, 64, seed=31)
    v[0, 1, 1, 3], v[0, 2, 0, 4], k[0, 5, 1, 63] = NAN, math.inf, -math.inf
    kc, vc = torch.zeros(2, 4, 2, 64, dtype=BF, device="cuda"), torch.zeros(2, 4, 2, 64, dtype=BF, device="cuda")
    kda.append_kv(k.cuda(), v.cuda(), kc, vc, torch.arange(6, device="cuda")[None].contiguous())
    assert torch.equal(kc.cpu().flatten(0, 1)[:6].view(torch.int16), k[0].view(torch.int16))
    assert torch.equal(vc.cpu().flatten(0, 1)[:6].view(torch.int16), v[0].view(torch.int16))
    assert not kc.flatten(0, 1)[6:].any() and not vc.flatten(0, 1)[6:].any()


# ---------------------------------------------------------------------------
# paged_attention
# ---------------------------------------------------------------------------

def case(lengths, Hq, Hk, D, page, seed, layout="tokens", spare=2, width=None):
    """q, caches, table and lengths on the CPU (caches on the GPU as laid out); unused entries name no page, and
    what no token of a sequence lies in is NaN."""
    n = len(lengths)
    used = [-(-max(0, x) // page) for x in lengths]
    width = width or max(1, max(used))
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((n, width), -1, dtype=torch.int32)
    kc, vc = caches(layout, pages, page, Hk, D, seed + 1)
    dirty = torch.ones(pages, page, dtype=torch.bool)
    at = 0
    for i, x in enumerate(lengths):
        table[i, :used[i]] = order[at:at + used[i]].int()
        for j in range(used[i]):
            dirty[table[i, j], :min(page, x - j * page)] = False
        at += used[i]
    kc[dirty.cuda()] = NAN
    vc[dirty.cuda()] = NAN
    return rand(n, Hq, D, seed=seed + 3), kc, vc, table, torch.tensor(lengths, dtype=torch.int32)


def attend(q, kc, vc, table, lengths, scale, window=None):
    out = torch.full(q.shape, NAN, dtype=BF, device="cuda")
    lse = torch.full(q.shape[:2], NAN, dtype=torch.float32, device="cuda")
    kda.paged_attention(q.cuda(), kc, vc, table.cuda(), lengths.cuda(), out, scale, lse=lse, window=window)
    return out, lse


def hold(q, kc, vc, table, lengths, scale, window=None):
    out, lse = attend(q, kc, vc, table, lengths, scale, window)
    wo, wl, bo, bl = ref.attention(q, kc.cpu(), vc.cpu(), table, lengths, scale, window)
    check("out", out, wo, bo)
    check("lse", lse, wl, bl)
    return out, lse


@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 16), (4, 4, 64), (8, 1, 128), (32, 4, 128), (6, 2, 48), (5, 1, 96), (40, 2, 128),
                                     (34, 2, 80), (16, 16, 32), (2, 1, 256), (3, 3, 192), (16, 2, 112), (9, 3, 160),
                                     (12, 2, 224)])
def test_attention_heads(Hq, Hk, D):
    hold(*case([1, 33, 0, 300], Hq, Hk, D, 16, D + Hq), D ** -0.5)


@pytest.mark.parametrize("page", [1, 3, 16, 100, 128, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads", "woven"])
def test_attention_pages(page, layout):
    hold(*case([1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 0, 700], 4, 2, 64, page, page, layout), 0.125)


@pytest.mark.parametrize("lengths", [[5000], [1, 5000, 0, 2049], [256] * 3, [2560, 2561, 2559, 2688, 2687]])
def test_attention_splits(lengths):
    hold(*case(lengths, 8, 2, 128, 64, len(lengths), width=100), 128 ** -0.5)


@pytest.mark.parametrize("window", [1, 31, 300, 4096])
def test_attention_window(window):
    hold(*case([1, 30, 299, 300, 301, 3000, 0], 4, 2, 64, 16, window), 0.125, window)


def test_attention_sharp_and_flat_scores():
    """One token that takes all the weight, early, late and in another split; equal scores; tiny and negative scales."""
    q, kc, vc, table, lengths = case([900, 900, 900, 900], 4, 1, 64, 16, 77)
    for i, t in enumerate((0, 450, 899)):
        kc[table[i, t // 16], t % 16, 0] = (q[i, 0] * 30).cuda()
    hold(q, kc, vc, table, lengths, 0.125)
    hold(q, kc, vc, table, lengths, 0.0)
    hold(q, kc, vc, table, lengths, -0.01)


def test_attention_bad_pages_and_lengths():
    """Pages outside the cache are not read, their tokens not visible; lengths beyond the table are cut."""
    q, kc, vc, table, lengths = case([200, 200, 200, 64], 4, 2, 64, 16, 88)
    table[0, 3], table[0, 12], table[1, :] = -7, 1 << 30, -1
    table[2, 5] = kc.shape[0]
    lengths[3] = 1 << 30
    table[3, 4:] = -1
    out, lse = hold(q, kc, vc, table, lengths, 0.125)
    assert not out[1].any() and torch.isinf(lse[1]).all()
    lengths[:] = -5
    out, lse = hold(q, kc, vc, table, lengths, 0.125)
    assert not out.any() and torch.isinf(lse).all()


def test_attention_non_finite_inputs_stay_with_what_sees_them():
    q, kc, vc, table, lengths = case([200, 200, 200], 4, 2, 64, 16, 99)
    clean, clean_lse = attend(q, kc, vc, table, lengths, 0.125)
    kc[table[0, 2], 3, 1, 7] = NAN
    vc[table[1, 4], 2, 0, 9] = math.inf
    out, lse = attend(q, kc, vc, table, lengths, 0.125)
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.equal(lse[0, :2], clean_lse[0, :2])
    assert torch.isinf(out[1, :2, 9]).all()
    rest = torch.ones(64, dtype=torch.bool, device="cuda")
    rest[9] = False
    assert torch.equal(out[1, :2][:, rest], clean[1, :2][:, rest]) and torch.equal(out[1, 2:], clean[1, 2:])
    assert torch.equal(out[2], clean[2])


def test_attention_strided_queries_and_tables():
    q, kc, vc, table, lengths = case([100, 40], 4, 2, 64, 16, 111)
    wide = torch.cat([rand(2, 1, 64, seed=1), q, rand(2, 3, 64, seed=2)], 1).cuda()
    tables = torch.cat([table, torch.full((2, 3), 5, dtype=torch.int32)], 1).cuda()
    out = torch.empty(2, 4, 64, dtype=BF, device="cuda")
    kda.paged_attention(wide[:, 1:5], kc, vc, tables[:, :table.shape[1]], lengths.cuda(), out, 0.125)
    same, _ = attend(q, kc, vc, table, lengths, 0.125)
    assert torch.equal(out, same)


def test_attention_empty_calls():
    q, kc, vc, table, lengths = case([10], 2, 1, 64, 16, 5)
    none = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    kda.paged_attention(none, kc, vc, table[:0].cuda(), lengths[:0].cuda(), torch.empty_like(none), 1.0)
    out = torch.full((1, 2, 64), NAN, dtype=BF, device="cuda")
    kda.paged_attention(q.cuda(), kc, vc, table[:, :0].cuda(), lengths.cuda(), out, 1.0)
    assert not out.any()
    kda.paged_attention(q.cuda(), kc[:0], vc[:0], table.cuda(), lengths.cuda(), out, 1.0)
    assert not out.any()


def test_attention_replays_from_a_graph():
    """Captured with its workspace; replays follow lengths that change on the device, with eager work between."""
    q, kc, vc, table, lengths = case([3000, 2000], 8, 2, 64, 16, 123)
    gq, gt, gl = cuda(q, table, lengths)
    out, lse = torch.empty(2, 8, 64, dtype=BF, device="cuda"), torch.empty(2, 8, dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kda.paged_attention(gq, kc, vc, gt, gl, out, 0.125, lse=lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.paged_attention(gq, kc, vc, gt, gl, out, 0.125, lse=lse)
    for cut in (0, 7, 1500, 2999):
        gl.copy_((lengths - cut).clamp(min=0))
        want, want_lse = attend(q, kc, vc, table, (lengths - cut).clamp(min=0), 0.125)
        out.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_attention_on_two_streams():
    """Calls that may overlap share nothing."""
    a, b = case([4000, 100], 8, 2, 64, 16, 131), case([200, 3900], 8, 2, 64, 16, 141)
    want = [attend(*x, 0.125) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [[t.cuda() for t in x] for x in (a, b)]
    torch.cuda.synchronize()
    outs = [[] for _ in range(2)]
    for _ in range(20):
        for s, x, o in zip(streams, inputs, outs):
            with torch.cuda.stream(s):
                out, lse = torch.empty(2, 8, 64, dtype=BF, device="cuda"), torch.empty(2, 8, dtype=torch.float32, device="cuda")
                kda.paged_attention(*x[:1], x[1], x[2], x[3], x[4], out, 0.125, lse=lse)
                o.append((out, lse))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w[0], x) and torch.equal(w[1], y) for x, y in o)


def test_a_long_cache_past_32_bits():
    """A cache of 5 GiB: pages whose offsets pass 2^32 bytes and 2^31 elements."""
    pages, page, Hk, D = 1 << 15, 128, 5, 128
    kc = torch.zeros(pages, page, Hk, D, dtype=BF, device="cuda")
    vc = torch.zeros(pages, page, Hk, D, dtype=BF, device="cuda")
    far = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    k, v = rand(1, 300, Hk, D, seed=1), rand(1, 300, Hk, D, seed=2)
    t = torch.arange(300)
    slots = (far[0].long()[t // page] * page + t % page)[None].contiguous()
    kda.append_kv(k.cuda(), v.cuda(), kc, vc, slots.cuda())
    near = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    small_k, small_v = kc[far[0].long().cuda()].cpu(), vc[far[0].long().cuda()].cpu()
    assert torch.equal(small_k.flatten(0, 1)[:300], k[0]) and torch.equal(small_v.flatten(0, 1)[:300], v[0])
    q = rand(1, 10, D, seed=3)
    lengths = torch.tensor([300], dtype=torch.int32)
    out, lse = attend(q, kc, vc, far, lengths, D ** -0.5)
    wo, wl, bo, bl = ref.attention(q, small_k, small_v, near, lengths, D ** -0.5)
    check("out", out, wo, bo)
    check("lse", lse, wl, bl)


def test_rotary_of_more_than_2_to_31_elements():
    T, H, D = (1 << 17) + 40, 32, 512
    q = torch.empty(1, T, H, D, dtype=BF, device="cuda")
    q[:, -64:] = rand(1, 64, H, D, seed=1).cuda()
    q[:, :-64] = 1.0
    pos = torch.arange(T, device="cuda")[None]
    f, w = freqs(64).cuda(), rand(D, seed=2).cuda()
    out = torch.full_like(q, NAN)
    kda.qk_norm_rotary(q, None, pos, f, out, None, w)
    tail = torch.full((1, 64, H, D), NAN, dtype=BF, device="cuda")
    kda.qk_norm_rotary(q[:, -64:], None, pos[:, -64:].contiguous(), f, tail, None, w)
    assert torch.equal(out[:, -64:], tail)
    check("q", tail, *ref.rotary(q[:, -64:].cpu(), pos[:, -64:].cpu(), f.cpu(), w.cpu()))


# ---------------------------------------------------------------------------
# tables for many tokens: a wave a split
# ---------------------------------------------------------------------------

WIDE = 1 << 18  # tokens that a table has room for


@pytest.mark.parametrize("Hq,Hk,D", [(2, 2, 16), (4, 4, 64), (16, 2, 128), (6, 2, 48), (10, 2, 96), (40, 2, 128),
                                     (34, 2, 80), (16, 16, 32), (4, 2, 256), (3, 3, 192), (9, 3, 160), (12, 2, 224)])
def test_attention_wide_tables_heads(Hq, Hk, D):
    hold(*case([1, 33, 0, 1300], Hq, Hk, D, 16, D + Hq, width=WIDE // 16), D ** -0.5)


@pytest.mark.parametrize("page", [1, 3, 100, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads", "woven"])
def test_attention_wide_tables_pages(page, layout):
    hold(*case([1, 31, 32, 127, 128, 129, 191, 192, 193, 385, 0, 700], 4, 2, 64, page, page, layout, width=WIDE // page), 0.125)


@pytest.mark.parametrize("lengths", [[5000, 0], [1, 30000, 0, 2049], [384] * 3, [191, 192, 193, 383, 384, 385]])
@pytest.mark.parametrize("window", [None, 130, 200000])
def test_attention_wide_tables_splits(lengths, window):
    hold(*case(lengths, 8, 4, 128, 64, len(lengths), width=WIDE // 64), 128 ** -0.5, window)


def test_attention_wide_tables_bad_pages_and_values():
    q, kc, vc, table, lengths = case([900, 900, 900, 64], 4, 2, 64, 16, 188, width=WIDE // 16)
    table[0, 3], table[0, 32], table[1, :] = -7, 1 << 30, -1
    table[2, 5] = kc.shape[0]
    lengths[3] = 1 << 30  # as far as the table goes, whose other pages are none
    out, lse = hold(q, kc, vc, table, lengths, 0.125)
    assert not out[1].any() and torch.isinf(lse[1]).all()
    kc[table[0, 2], 3, 1, 7] = NAN
    vc[table[2, 4], 2, 0, 9] = math.inf
    bad, bad_lse = attend(q, kc, vc, table, lengths, 0.125)
    assert bad[0, 2:].isnan().all() and bad_lse[0, 2:].isnan().all() and torch.isinf(bad[2, :2, 9]).all()
    assert torch.equal(bad[0, :2], out[0, :2]) and torch.equal(bad[1], out[1]) and torch.equal(bad[2, 2:], out[2, 2:])


@pytest.mark.parametrize("Hq,Hk,D", [(4, 2, 16), (4, 1, 48), (8, 2, 144), (17, 1, 192), (4, 4, 256)])
def test_attention_splits_of_other_widths(Hq, Hk, D):
    hold(*case([5000, 1, 0, 2049, 512, 513], Hq, Hk, D, 64, D, width=100), D ** -0.5)
