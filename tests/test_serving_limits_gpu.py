"""Serving operators at the ends of their ranges: scores and value scales of extreme size, and
lengths that are out of range."""
import math

import pytest

import serving_ref as ref
from test_serving_gpu import A, BF, Cache, ints, normal, scattered, sums  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# Longest history in positions: a CTA a segment, a cluster a segment, runs of tiles and their join.
PATHS = [[200], [700, 90], [9000, 30]]


# ------------------------------------------------------------- large scores
@pytest.mark.parametrize("d,G,n_q", [(64, 1, 1), (128, 4, 1), (64, 4, 3), (128, 4, 5), (64, 8, 4)])
@pytest.mark.parametrize("lens", PATHS)
@pytest.mark.parametrize("top", [2.0 ** 24 + 2, 2.0 ** 25 + 100, 2.0 ** 26, 2.0 ** 27 + 512, -(2.0 ** 25) - 100])
def test_decode_scores_beyond_the_exponent(A, top, lens, d, G, n_q):
    """The largest score in base 2 is `top`, where FP32 no longer holds whole numbers: three keys of equal
    score far above all others take the weight.  Their value rows are equal and their scale is a power of
    two, so O is that row exactly (a BF16 number: 7 bits and a power of two), whatever the roundings of the
    weights' sum."""
    page, Hkv = 32, 2
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    c.codes[0][:] = 0
    c.codes[0][..., 0] = 60 if top > 0 else -127
    c.scales[0][:] = abs(top) / 100 * 2.0 ** -10
    c.scales[1][:] = 0.25
    row = torch.randint(-127, 128, (Hkv, d), generator=torch.Generator().manual_seed(1), dtype=torch.int8)
    for b, n in enumerate(lens):
        for pos in (3, (n - n_q) // 2, n - n_q):  # visible to every row
            p = tables[b][pos // page]
            c.codes[0][p, :, pos % page, 0] = 100 if top > 0 else -100
            c.codes[1][p, :, pos % page] = row
    c.upload()
    q = torch.zeros((len(lens), n_q, Hkv * G, d), dtype=BF)
    q[..., 0] = 2.0 ** 10
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens), scale=math.log(2.0))
    A.attn_check_status()
    want = (row.double() * 0.25).repeat_interleave(G, 0)
    assert (o.cpu().double() == want).all()
    # Nine roundings of 2^-24: the page's scale, the call's, log2 e, their product, that times the page's
    # scale, the score, its sum with log2 3, ln 2, the last product; and log2 3 < 1.6 beside 2^24 and more.
    assert ((lse.cpu().double() / (top * math.log(2.0)) - 1).abs() <= (9 + 1.6) * 2.0 ** -24 + 2.0 ** -40).all()


# ------------------------------------------------------------- value scales
def check_weighted(c, q, lens, scale, o, lse):
    """The bound of a weight's rounding follows the row's own weighted values: with P_j the row's exact
    softmax, weights P vs are FP16, relative 2^-11, as p 2^15 vs / R, and where that falls below 2^-14,
    absolute 2^-25, i.e. 2^-40 R.  Either every scale that the row's warp has met is at least 2^-8 R, so that
    the key of its largest p, which is 1 there, has a weight of 2^-8 R; or R is the row's own: at most twice
    its largest weight, or, from the time before, 2^8 of it.  So R is below 2^9 times the row's largest
    P_j vs_j, whatever the scales of pages that the row does not see or barely weighs, and a key is off by
    at most 2^-31 * 127 of that."""
    B, n_q, H, d = q.shape
    Hkv, page = c.codes[0].shape[1], c.codes[0].shape[2]
    G = H // Hkv
    o, lse = o.cpu(), lse.cpu()
    for b, n in enumerate(lens):
        k, v = c.values(0, b, n), c.values(1, b, n)
        last = torch.tensor([n - n_q + i for i in range(n_q) for _ in range(G)])
        ids = c.tables[b][:-(-n // page)]
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            qr = q[b, :, hs].reshape(-1, d)
            r, rl, a, size = ref.attention(qr, k[:, h], v[:, h], scale, last)
            vs = c.scales[1][ids, h].double().repeat_interleave(page)[:n]
            s = torch.where(torch.arange(n)[None] <= last[:, None], scale * (qr.double() @ k[:, h].t()), -torch.inf)
            p = torch.exp(s - torch.where(rl.isinf(), 0.0, rl)[:, None])
            least = n * 127 * 2.0 ** -31 * (p * vs).amax(-1)[:, None]
            got, gl = o[b, :, hs].reshape(-1, d).double(), lse[b, :, hs].reshape(-1).double()
            bound = ref.output_bound(r, a, size, d, 2.0 ** -11) + least
            assert ((got - r).abs() <= bound).all(), (b, h)
            live = ~rl.isinf()
            assert (got[~live] == 0).all() and (gl[~live] == -torch.inf).all()
            assert ((gl - rl)[live].abs() <= ref.lse_bound(rl, size, d)[live]).all(), (b, h)


ROWS = [(64, 1, 1), (128, 4, 1), (64, 4, 3), (128, 4, 3), (128, 4, 5), (64, 5, 4), (128, 8, 4)]


@pytest.mark.parametrize("d,G,n_q", ROWS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("lens", PATHS)
def test_decode_value_scales_of_every_ratio(A, lens, page, d, G, n_q):
    """Value scales spread over 2^90 from page to page, and scores over some tens: the row's weight lies on
    pages of any scale."""
    Hkv = 2
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    g = torch.Generator().manual_seed(len(lens) + page)
    c.scales[1] *= 2.0 ** torch.randint(-45, 46, c.scales[1].shape, generator=g)
    c.scales[1][tables[0][1]] = 0
    c.upload()
    q = normal((len(lens), n_q, Hkv * G, d), 1) * 2
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    check_weighted(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d,G,n_q", [r for r in ROWS if r[2] > 1])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("long", [1, 5, 70])
def test_decode_large_values_of_later_tokens(A, long, page, d, G, n_q):
    """The newest token opens a page whose value scale is 2^45 times the others': the tokens before it, which
    must not see it, keep their precision; the newest one sees it.  In a tile's second half where the page is 16."""
    Hkv = 2
    lens = [page * long + 1, page * (long + 1) + 1]
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    for t in tables:
        c.scales[1][t[-1]] *= 2.0 ** 45
    c.upload()
    q = normal((2, n_q, Hkv * G, d), 1)
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    check_weighted(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d,G,n_q", ROWS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("lens", PATHS)
def test_decode_large_values_of_no_weight(A, lens, page, d, G, n_q):
    """Every third page holds values 2^45 times as large as the others', behind keys whose weights are about
    2^-90 of the row's largest: they change nothing that can be seen."""
    Hkv = 2
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    c.codes[0][..., 0] = 0
    for t in tables:
        for p in t[1::3]:
            c.scales[1][p] *= 2.0 ** 45
            c.codes[0][p, ..., 0] = -127
    c.scales[0][:] = 0.01
    c.upload()
    q = normal((len(lens), n_q, Hkv * G, d), 1)
    q[..., 0] = 49.0  # -127 * 0.01 * 49 = -62 = -90 ln 2
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens), scale=1.0)
    A.attn_check_status()
    check_weighted(c, q, lens, 1.0, o, lse)


# ------------------------------------------------------------------ lengths
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_append_of_lengths_out_of_range_leaves_the_cache(A, d, few):
    """A sequence whose start is negative, or whose rows begin before the input, end behind it or run
    backwards, is left out: what its pages hold stays as it is.  The others are written."""
    page, Hkv, T = 16, 3, 12 if few else 64
    tables = [[0, 1, 8, 9], [2, 3, 10, 11], [4, 5, 6, 7]]
    rows = [normal((T, Hkv, d), 1), normal((T, Hkv, d), 2)]
    gpu_rows = [x.cuda() for x in rows]
    for cu, starts, good in (([0, 4, 8, T], [-1, 0, 5], (1, 2)), ([0, 4, 8, T], [3, -2 ** 31, 0], (0, 2)),
                             ([-4, 4, 8, T], [0, 0, 0], (1, 2)), ([0, 4, 8, T + 1], [0, 2, 0], (0, 1)),
                             ([0, 9, 4, T], [0, 0, 0], (0, 2)), ([0, 4, 2 ** 31 - 1, T], [0, 0, 0], (0,)),
                             ([-2 ** 31, -1, 4, T], [0, 0, 3], (2,))):
        c = Cache(12, Hkv, page, d, tables)
        for b in good:
            for i in range(2):
                ref.append(rows[i][cu[b]:cu[b + 1]], c.codes[i], c.scales[i], tables[b], starts[b])
        A.attn_cache_append_int8(*gpu_rows, *c.gpu, ints(cu), ints(starts))
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
        assert c.equal(), (cu, starts)
    A.attn_check_status()


def test_read_reports_lengths_out_of_range(A):
    """Lengths that do not begin at 0, end at T and rise are reported, also where every token of the output
    has a page."""
    page, d, Hkv = 16, 64, 2
    c = Cache(12, Hkv, page, d, [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]])
    for cu, T in (([-3, 20, 40], 40), ([0, 20, 41], 40), ([0, 40, 30], 40), ([0, 40, 39], 40), ([2, 20, 40], 40)):
        A.attn_cache_read_int8(*c.gpu, ints(cu), ints([0, 0]), T)
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
    A.attn_cache_read_int8(*c.gpu, ints([0, 20, 40]), ints([0, 0]), 40)
    A.attn_check_status()


def test_status_of_several_calls_at_once(A):
    """Reports of several calls since the last check are given together and cleared together."""
    page, d, Hkv = 16, 64, 2
    c = Cache(4, Hkv, page, d, [[0, 1]])
    rows, q = normal((4, Hkv, d), 1).cuda(), normal((1, 1, 4, d), 2).cuda()
    for _ in range(2):
        A.attn_varlen_plan(ints([0, 9]), 4, 4, Hkv)
        A.attn_cache_append_int8(rows, rows, *c.gpu, ints([0, 4]), ints([-1]))
        A.attn_decode_int8(q, *c.gpu, ints([99]))
        with pytest.raises(A.AttnError, match=r"varlen [1-9]\d*, cache [1-9]\d*, decode [1-9]"):
            A.attn_check_status()
        A.attn_check_status()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,d", [((4, 1), 64), ((2, 2), 128)])
@pytest.mark.parametrize("lens", [[700], [300] * 40])
@pytest.mark.parametrize("top", [2.0 ** 24 * 1.5625, 2.0 ** 28 * 1.40625, 2.0 ** 31 * 1.9375, 2.0 ** 33 * 1.0546875, 2.0 ** 60,
                                 -(2.0 ** 34) * 1.15625])
def test_prompt_scores_beyond_the_exponent(A, top, lens, heads, d, causal):
    """Up to three keys of the same largest score far above all others, of the same value row: O is that row
    and LSE the score plus the logarithm of the keys' number."""
    H, Hkv = heads
    T, cu = sum(lens), sums(lens)
    q, k, v = torch.zeros((T, H, d), dtype=BF), torch.zeros((T, Hkv, d), dtype=BF), normal((T, Hkv, d), 3)
    q[..., 0] = 2.0 ** 10
    k[..., 0] = top * 2.0 ** -10 * (0.5 if top > 0 else 2.0)
    row, seen = normal((Hkv, d), 4), torch.zeros(T)
    for b, n in enumerate(lens):
        for pos in (0, n // 2, n - 1):
            k[cu[b] + pos, :, 0], v[cu[b] + pos] = top * 2.0 ** -10, row
            seen[cu[b] + (pos if causal else 0):cu[b + 1]] += 1
    plan = A.attn_varlen_plan(ints(cu), T, H, Hkv, causal=causal)
    o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan, scale=1.0, causal=causal)
    A.attn_check_status()
    want = row.double().repeat_interleave(H // Hkv, 0)
    # P is rounded to BF16 (2^-8), and so is O; 2^-18 for the FP32 sums, the exponential and the division.
    assert ((o.cpu().double() - want).abs() <= (2.0 ** -7 + 2.0 ** -15) * want.abs()).all()
    # In units of 2^-24 of the score: the maximum's product with log2 e, by which all weights of a row may be
    # off together, log2 e itself, the maximum's product with the scale, the logarithm's sum, and ln 3 < 1.1
    # beside 2^24; 2^-18 for the logarithm.
    exact = top + torch.log(seen.double())[:, None]
    assert ((lse.cpu().double() - exact).abs() <= 6 * 2.0 ** -24 * abs(top) + 2.0 ** -18).all()


@pytest.mark.parametrize("d,G", [(64, 1), (128, 2)])
@pytest.mark.parametrize("page,lens", [(32, [300, 470]), (16, [2000, 280]), (64, [9000, 290])])
@pytest.mark.parametrize("big,small", [(40, -10), (-10, 40), (100, -100)])
def test_decode_rows_that_see_nothing_of_a_warp(A, big, small, page, lens, d, G):
    """256 newest tokens: a warp has tiles of which the first ones see nothing, and the value scales of
    these differ by 2^50 and more."""
    Hkv, n_q = 1, 256
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    for t in tables:
        for j, p in enumerate(t):
            c.scales[1][p] *= 2.0 ** (big if j * page // 128 % 2 == 0 else small)
    c.upload()
    q = normal((2, n_q, Hkv * G, d), 1)
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    check_weighted(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d,G", [(64, 4), (128, 4)])
@pytest.mark.parametrize("jump", [100.0, 150.0])
@pytest.mark.parametrize("big", [40, 100])
def test_decode_maximum_that_leaps(A, big, jump, d, G):
    """The score's maximum leaps by more or less than FP32's exponents hold where the value scale falls by
    2^60 to 2^200: what was summed before counts as long as its weights do."""
    Hkv, page, lens = 1, 32, [500, 1500]
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    c.codes[0][..., 0] = 0
    c.scales[0][:] = 0.01
    for t in tables:
        for j, p in enumerate(t):
            c.scales[1][p] *= 2.0 ** (big if j < 4 else -20 if big == 40 else -100)
            if j >= 4:
                c.codes[0][p, ..., 0] = 100
    c.upload()
    q = normal((2, 1, Hkv * G, d), 1)
    q[..., 0] = jump  # times 100 * 0.01
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens), scale=math.log(2.0))
    A.attn_check_status()
    assert o.isfinite().all()
    if jump < 126 or big == 40:  # else weights of p < 2^-126, which count as 0, would matter
        check_weighted(c, q, lens, math.log(2.0), o, lse)


@pytest.mark.parametrize("d,G", [(64, 1), (64, 4), (128, 4), (128, 20)])
@pytest.mark.parametrize("lens", [[500, 200], [1500, 300], [9000, 2000], [3000] * 40])
def test_decode_small_weights_of_large_values(A, lens, d, G):
    """The first 128 positions have weights of about 2^-118 of the row's largest and value scales 2^140 times
    the others': O is theirs, whichever way warps and parts are joined."""
    Hkv, page = 1, 32
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    c.codes[0][..., 0] = 0
    c.scales[0][:] = 0.002
    for t in tables:
        for j, p in enumerate(t):
            c.scales[1][p] *= 2.0 ** (100 if j < 4 else -40)
            if j >= 4:
                c.codes[0][p, ..., 0] = 100
    c.upload()
    q = normal((len(lens), 1, Hkv * G, d), 1)
    q[..., 0] = 592.0  # 100 * 0.002 * 592 = 118.4
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens), scale=math.log(2.0))
    A.attn_check_status()
    check_weighted(c, q[:3], lens[:3], math.log(2.0), o[:3], lse[:3])
