"""paged_attention at the limits of its numbers and places: the largest scales and
scores, infinite ones, more queries than a join takes, caches at odd elements (and
append_kv's), on every way through the kernels: one split, splits shared by a
workgroup's waves, a wave a split, joins of few and of many splits."""
import math

import pytest
import torch

import gated_delta_rule_36_amd as kda
import mixer_ref as ref
from mixer_ref import check
from test_attention_gpu import WIDE, attend, case, freqs, rand

pytestmark = pytest.mark.gpu

# (lengths, key heads, channels, tokens that the table has room for)
WAYS = [([5, 200, 0], 2, 64, 208), ([3000, 5, 0, 700], 2, 64, 3008), ([3000, 5], 2, 256, 3008),
        ([900, 5, 0, 193], 4, 128, WIDE), ([130, 2000], 4, 256, WIDE), ([20000, 9], 8, 64, WIDE),
        ([700, 0] + [3] * 62, 4, 64, 1 << 14), ([700, 0] + [3] * 62, 4, 144, 1 << 14)]


def build(lengths, Hk, D, room, seed):
    return case(lengths, 2 * Hk, Hk, D, 16, seed, width=-(-room // 16))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("scale", [3.3e38, -3.3e38])
def test_the_largest_scales_with_queries_of_zero(way, scale):
    """Every score is 0: the mean of the values, and the logarithm of the number of tokens."""
    q, kc, vc, table, lengths = build(*way, 211)
    q.zero_()
    out, lse = attend(q, kc, vc, table, lengths, scale)
    wo, wl, bo, bl = ref.attention(q, kc.cpu(), vc.cpu(), table, lengths, scale)
    check("out", out, wo, bo)
    check("lse", lse, wl, bl)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_up_to_the_largest_numbers(way, sign):
    """Scores of 1, 2 and 3 times 1e38, exact as they are formed: the tokens with the largest share the weight,
    the others' is 0, and the maximum is the logarithm of the sum."""
    q, kc, vc, table, lengths = build(*way, 221)
    q.zero_()
    q[..., 0] = 1.0
    pages, page = kc.shape[:2]
    seen = ~kc[..., 0, 0].isnan()
    level = torch.randint(1, 4, (pages, page), generator=torch.Generator().manual_seed(5)).cuda()
    kc[..., 0] = torch.where(seen, sign * level, math.nan)[..., None].to(kc.dtype)
    out, lse = attend(q, kc, vc, table, lengths, 1e38)
    # the same weights as of scores of 1, 2 and 3 times 1000, where exp(-1000) is 0 in 64 bits, too
    wo, wl, _, _ = ref.attention(q, kc.cpu(), vc.cpu(), table, lengths, 1000.0)
    # of n equal probabilities the sum, its reciprocal and the product are rounded, and the parts leave 2^-16; a
    # value is below 8 here.  The score is one product's rounding off, and so is its logarithm
    check("out", out, wo, torch.tensor(8 * (2.0 ** -16 + (max(way[0]) + 16) * ref.U32), dtype=torch.float64))
    check("lse", lse, 1e38 * torch.round(wl / 1000), torch.tensor(3e38 * 4 * ref.U32, dtype=torch.float64))


@pytest.mark.parametrize("way", WAYS)
def test_scores_of_minus_infinity(way):
    """Such tokens have no weight beside others; where every visible one is such there is no softmax: NaN, and a
    logarithm of -inf.  Zeros are of sequences without a visible token alone."""
    q, kc, vc, table, lengths = build(*way, 231)
    q[..., 0] = 1.0
    k0 = kc[..., 0].clone()
    # every other page, as a sequence's own run of pages: in the reference these pages are none
    part = table.clone()
    for n, length in enumerate(way[0]):
        used = -(-length // 16)
        for j in range(used):
            if used > 1 and j % 2 == 0:
                kc[table[n, j], ..., 0] = -math.inf
                part[n, j] = -1
    clean = kc.clone()
    clean[..., 0] = k0
    out, lse = attend(q, kc, vc, table, lengths, 0.125)
    wo, wl, bo, bl = ref.attention(q, clean.cpu(), vc.cpu(), part, lengths, 0.125)
    check("out", out, wo, bo)
    check("lse", lse, wl, bl)
    kc[..., 0] = -math.inf
    out, lse = attend(q, kc, vc, table, lengths, 0.125)
    some = (lengths > 0).cuda()
    assert out[some].isnan().all() and not out[~some].any()
    assert torch.equal(lse, torch.full_like(lse, -math.inf))
    table[0] = -1  # pages that are none: not visible
    out, lse = attend(q, kc, vc, table, lengths, 0.125)
    some[0] = False
    assert out[some].isnan().all() and not out[~some].any()
    assert torch.equal(lse, torch.full_like(lse, -math.inf))


@pytest.mark.parametrize("way", WAYS)
def test_scores_of_plus_infinity(way):
    """A key that is infinite where the query is positive: no softmax, but a sum, whose logarithm is infinite; NaN
    beside it leaves neither."""
    q, kc, vc, table, lengths = build(*way, 241)
    q[..., 0] = 1.0
    n = max(range(len(way[0])), key=lambda i: way[0][i])
    for t in {0, way[0][n] // 2, way[0][n] - 1}:
        clean, clean_lse = attend(q, kc, vc, table, lengths, 0.125)
        bad = kc.clone()
        bad[table[n, t // 16], t % 16, 1, 0] = math.inf
        out, lse = attend(q, bad, vc, table, lengths, 0.125)
        assert out[n, 2:4].isnan().all() and (lse[n, 2:4] == math.inf).all()
        out[n, 2:4], lse[n, 2:4] = clean[n, 2:4], clean_lse[n, 2:4]
        assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
        bad[table[n, (t + 1) % way[0][n] // 16], (t + 1) % way[0][n] % 16, 1, 3] = math.nan
        out, lse = attend(q, bad, vc, table, lengths, 0.125)
        assert out[n, 2:4].isnan().all() and lse[n, 2:4].isnan().all()


def test_more_queries_than_a_join_of_them_would_have_workgroups_for():
    """2^22 query heads of 128 channels: one split each, so nothing is joined."""
    q, kc, vc, table, lengths = case([1 + i % 16 for i in range(64)], 32, 1, 128, 16, 251)
    few, few_lse = attend(q, kc, vc, table, lengths, 0.125)
    n = 1 << 11
    out, lse = attend(q.repeat(n, 1, 1), kc, vc, table.repeat(n, 1), lengths.repeat(n), 0.125)
    assert (out.unflatten(0, (n, 64)) == few).all() and (lse.unflatten(0, (n, 64)) == few_lse).all()


def odd(t):
    """t's numbers at an odd element of wider rows, NaN between them."""
    room = torch.full((t.numel() // t.shape[-1] * (t.shape[-1] + 3) + 1,), math.nan, dtype=t.dtype, device="cuda")
    y = room[1:].view(*t.shape[:-1], t.shape[-1] + 3)[..., :t.shape[-1]]
    y.copy_(t)
    return room, y


@pytest.mark.parametrize("way", WAYS)
def test_caches_at_odd_places(way):
    q, kc, vc, table, lengths = build(*way, 261)
    out, lse = attend(q, kc, vc, table, lengths, 0.125)
    wide = torch.full((q.shape[0], q[0].numel() + 3), math.nan, dtype=q.dtype)
    wide[:, 1:-2] = q.flatten(1)
    queries = wide.cuda()[:, 1:-2].unflatten(1, q.shape[1:])
    again, again_lse = attend(queries, odd(kc)[1], odd(vc)[1], table, lengths, 0.125)
    assert torch.equal(again, out) and torch.equal(again_lse, lse)


@pytest.mark.parametrize("D,R", [(16, 8), (64, 64), (80, 20), (128, 32), (256, 256), (6, 2)])
def test_append_to_caches_at_odd_places(D, R):
    """The numbers of the call on contiguous caches, and nothing between the rows or behind the last is written."""
    k, v = rand(2, 7, 3, D, seed=1).cuda(), rand(2, 7, 3, D, seed=2).cuda()
    kc, vc = rand(5, 4, 3, D, seed=3).cuda(), rand(5, 4, 3, D, seed=4).cuda()
    slots = torch.randperm(20, generator=torch.Generator().manual_seed(5))[:14].view(2, 7).cuda()
    slots[1, 3] = -1
    positions, f, w = torch.arange(14, device="cuda").view(2, 7), freqs(R).cuda(), rand(D, seed=6).cuda()
    (kroom, ko), (vroom, vo) = odd(kc), odd(vc)
    for caches in ((kc, vc), (ko, vo)):
        kda.append_kv(k, v, *caches, slots, positions, f, w)
    for (room, got), want in (((kroom, ko), kc), ((vroom, vo), vc)):
        again, y = odd(want)
        assert torch.equal(got, want) and torch.equal(room.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("Hk,D,room", [(4, 16, 16), (4, 128, 16), (4, 64, WIDE), (2, 256, WIDE)])
def test_probabilities_keep_their_digits(Hk, D, room):
    """Four tokens whose values cancel to 2^-17 of their weighted sizes, so that out shows the probabilities' errors and
    not its own rounding.

    The scores are multiples of 1/8 up to 1 and exact, as are their differences.  A probability is off by 1.25 2^-24 of
    the multiplication with log2(e), 2^-23 of the exponential and 1.25 2^-23 of its parts; twelve products and their sums
    leave 12 2^-24, the sum of the probabilities, its reciprocal and the product with it 5 2^-24: 2^-19.5 in all.
    Probabilities good to 2^-16 are past it."""
    n = 16
    q, kc, vc, table, lengths = build([4] * n, Hk, D, room, 281)
    gen = torch.Generator().manual_seed(282)
    pick = lambda: torch.stack([torch.randperm(9, generator=gen)[:4] for _ in range(n * Hk)]).view(n, Hk, 4).transpose(1, 2)  # noqa: E731
    level = pick().double()  # [n, 4, Hk], each token's score times 8
    q.zero_()
    q[..., 0] = 1.0
    p = torch.softmax(level / 8, 1)[..., None]
    v = torch.randn(n, 4, Hk, D, generator=gen).clamp(-2, 2).to(q.dtype).double()
    v[:, 2:] = 0
    for t in (2, 3):  # what is left of the ones before, rounded
        v[:, t] = (-(p * v).sum(1) / p[:, t]).to(q.dtype).double()
    at = table[:, 0].long()
    kc[at, :4] = level[..., None].expand(n, 4, Hk, D).to(kc.dtype).cuda()
    vc[at, :4] = v.to(vc.dtype).cuda()
    out, lse = attend(q, kc, vc, table, lengths, 0.125)
    want = (p * v).sum(1).repeat_interleave(2, 1)
    size = (p * v.abs()).sum(1).repeat_interleave(2, 1)
    assert (want.abs() <= 2.0 ** -16 * size).double().mean() > 0.9
    check("out", out, want, 2.0 ** -19.5 * size)
    check("lse", lse, torch.logsumexp(level / 8, 1).repeat_interleave(2, 1), torch.tensor(2.0 ** -20, dtype=torch.float64))
