"""Attention over a prefix that a batch shares, against its plain 64-bit form."""
import math

import pytest

import serving_ref as ref
from test_serving_gpu import A, BF, Cache, ints, normal, scattered, sums  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def make(n0, lens, Hkv, page, d, seed=0, width=None):
    """A cache with the pages of the sequences and of the prefix; the prefix's pages."""
    tables, pages = scattered([-(-n0 // page)] + [-(-n // page) for n in lens], seed + 7)
    return Cache(pages, Hkv, page, d, tables[1:], seed=seed, width=width), tables[0] or [0]


# Which kernels read the prefix follows from the room in its table: as wide as it needs (one launch, the prefix read
# once a sequence, for the small ones here), or so wide that it is read once for 256 rows.
WIDE = 1 << 23
WIDTHS = pytest.mark.parametrize("room", [0, WIDE])


def call(A, q, c, pre, n0, lens, room=0, **kw):  # noqa: N803
    pre = pre + [-1] * (room // c.codes[0].shape[2])
    return A.attn_decode_shared_int8(q, *c.gpu[:4], ints(pre), ints([n0]), c.gpu[4], ints(lens), **kw)


def check(c, pre, n0, q, lens, scale, o, lse, shown=None):
    """Within the bounds of attn_decode_int8's tests: weights in FP16, those below 2^-20 of a part's largest off by
    2^-31 of it, times a code of 127.  A part's largest is no larger than the row's.  A weight e^(s - max s) below
    2^-126, the least normal FP32, counts as 0 or loses bits, as attn.h says: what such keys add to O is off by no more
    than itself (test_small_weights_of_large_values has rows of two keys whose weights are 2^-118 times e^(-9))."""
    B, n_q, H, d = q.shape
    Hkv, page = c.codes[0].shape[1], c.codes[0].shape[2]
    G = H // Hkv
    o, lse = o.cpu(), lse.cpu()
    k0, v0 = (ref.cached(c.codes[i], c.scales[i], pre, n0) for i in range(2))
    ids0 = torch.tensor(list(pre[:-(-n0 // page)]), dtype=torch.long).repeat_interleave(page)[:n0]
    for b, n in enumerate(lens):
        if shown is not None and b not in shown:
            continue
        k, v = torch.cat([k0, c.values(0, b, n)]), torch.cat([v0, c.values(1, b, n)])
        last = torch.tensor([n0 + max(n - n_q + i, -1) for i in range(n_q) for _ in range(G)])
        ids = torch.cat([ids0, torch.tensor(c.tables[b][:-(-n // page)], dtype=torch.long).repeat_interleave(page)[:n]])
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            qr = q[b, :, hs].reshape(-1, d)
            r, rl, a, size = ref.attention(qr, k[:, h], v[:, h], scale, last)
            vs = c.scales[1][ids, h].double()
            s = torch.where(torch.arange(len(k))[None] <= last[:, None], scale * (qr.double() @ k[:, h].t()), -torch.inf)
            p = torch.exp(s - torch.where(rl.isinf(), 0.0, rl)[:, None])
            least = len(k) * 127 * 2.0 ** -31 * ((p * vs).amax(-1)[:, None] if len(k) else 0.0)
            if len(k):
                tiny = torch.exp(s - s.amax(-1, keepdim=True)) < 2.0 ** -126
                least = least + torch.where(tiny, p, 0.0) @ v[:, h].abs()
            got, gl = o[b, :, hs].reshape(-1, d).double(), lse[b, :, hs].reshape(-1).double()
            bound = ref.output_bound(r, a, size, d, 2.0 ** -11) + least
            assert ((got - r).abs() <= bound).all(), (b, h, ((got - r).abs() / bound).max())
            live = ~rl.isinf()
            assert (got[~live] == 0).all() and (gl[~live] == -torch.inf).all()
            assert ((gl - rl)[live].abs() <= ref.lse_bound(rl, size, d)[live]).all(), (b, h)


LENS = [0, 1, 2, 15, 16, 17, 64, 130]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n0", [0, 1, 127, 128, 129, 1000])
@pytest.mark.parametrize("heads,n_q", [((2, 2), 1), ((14, 2), 2), ((12, 3), 5), ((64, 1), 1)])
@WIDTHS
def test_shared(A, room, heads, n_q, n0, page, d):
    """One row tile and two, full and ragged (8 to 512 rows a key head); sequences with less than n_q positions."""
    H, Hkv = heads
    c, pre = make(n0, LENS, Hkv, page, d)
    q = normal((len(LENS), n_q, H, d), 1)
    o, lse = call(A, q.cuda(), c, pre, n0, LENS, room)
    A.attn_check_status()
    check(c, pre, n0, q, LENS, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,G,n_q", [(1, 1, 1), (1, 1, 127), (1, 1, 128), (1, 1, 129), (1, 1, 255), (1, 1, 256), (3, 1, 86),
                                     (5, 4, 13), (3, 3, 29), (3, 5, 33), (2, 64, 5)])
@WIDTHS
def test_rows(A, room, B, G, n_q, d):
    """Rows at the tiles' and units' borders: the last unit with one tile behind units with two, and with both."""
    Hkv, page, n0, lens = 2, 32, 700, [n_q + 5 * b for b in range(B)]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, n_q, Hkv * G, d), 1)
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,n0", [(1, 1, 1, 100000), (40, 8, 8, 5000), (9, 64, 2, 30001), (80, 16, 4, 2500),
                                        (300, 7, 1, 6000)])
def test_long_prefixes(A, B, H, Hkv, n0, d):
    """Units in one, a few and many runs; several units a run."""
    page, lens = 64, [1 + 37 * b % 90 for b in range(B)]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, 1, H, d), 1)
    o, lse = call(A, q.cuda(), c, pre, n0, lens)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse, shown=(0, 1, B // 2, B - 1))


@pytest.mark.parametrize("width", [2, 40, 300])
@WIDTHS
def test_own_histories(A, room, width):
    """The own part in each of its forms (a CTA a segment, clusters, runs), ragged."""
    H, Hkv, d, page, n0 = 8, 2, 128, 32, 500
    lens = [min(n, width * page) for n in (9000, 1, 0, 700, 33, 5000)]
    c, pre = make(n0, lens, Hkv, page, d, width=width)
    q = normal((len(lens), 2, H, d), 1)
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("B,Hkv,G,n_q", [(70, 8, 4, 1), (90, 12, 1, 1), (45, 8, 4, 5), (300, 2, 7, 2)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("longest", [1500, 2100])
@WIDTHS
def test_many_ragged_histories(A, room, longest, B, Hkv, G, n_q, d, page):
    """About as many segments as CTAs, on both sides of the length up to which they are not split."""
    lens = [longest, 0, 1] + [(b * b * 13) % longest if b % 5 == 0 else (b * 31) % 90 for b in range(B - 3)]
    c, pre = make(700, lens, Hkv, page, d)
    q = normal((B, n_q, Hkv * G, d), 1)
    o, lse = call(A, q.cuda(), c, pre, 700, lens, room)
    A.attn_check_status()
    check(c, pre, 700, q, lens, 1 / math.sqrt(d), o, lse, shown=(0, 1, 2, 8, 33, B - 1))


def test_without_the_tensor_binding(A, monkeypatch):
    from precision_numerics_gb300 import attn

    lens = [9, 60]
    c, pre = make(300, lens, 2, 16, 64)
    q = normal((2, 1, 8, 64), 1).cuda()
    want = call(A, q, c, pre, 300, lens, WIDE)
    monkeypatch.setattr(attn, "_BINDING", attn._NoBinding)
    got = call(A, q, c, pre, 300, lens, WIDE)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    call(A, q, c, pre, 300, lens, WIDE, o=o, lse=lse)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(ValueError):
        call(A, q, c, pre, 300, lens, o=o.cpu())
    A.attn_check_status()


@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("B,G,n_q", [(80, 4, 16), (40, 8, 33), (170, 64, 1), (80, 2, 200)])
@pytest.mark.parametrize("n0", [0, 40, 1000])
def test_many_new_tokens(A, n0, B, G, n_q, d, page):
    """64 rows a sequence and key head and more, of many sequences: own positions by units of 256 rows; sequences of
    fewer positions than new tokens, of none, with a page that is not there and a length out of range."""
    Hkv = 2 if B < 160 else 1
    lens = [(n_q + 37 * b) % 400 for b in range(B)]
    lens[3], lens[4], lens[5] = 0, 1, max(1, n_q - 1)
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, n_q, Hkv * G, d), 1)
    o, lse = call(A, q.cuda(), c, pre, n0, lens)
    A.attn_check_status()
    scale = 1 / math.sqrt(d)
    check(c, pre, n0, q, lens, scale, o, lse, shown=(0, 3, 4, 5, 9, B - 1))
    again = call(A, q.cuda(), c, pre, n0, lens)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    at = next(b for b in range(10, B) if lens[b] > page)
    c.gpu[4][at, 0] = c.codes[0].shape[0]
    wrong = list(lens)
    wrong[7] = -5
    o, lse = call(A, q.cuda(), c, pre, n0, wrong)
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    wrong[7] = 0
    check(c, pre, n0, q, wrong, scale, o, lse, shown=(0, 7, at - 1))
    # As if the page's codes were in the prefix's place: only the rest of the sequence is seen.
    n = lens[at] - page
    part, part_lse = call(A, q[at:at + 1].cuda(), _Only(c, at), pre, n0, [n])
    A.attn_check_status()
    # Both within 2^-8 of a value for its rounding and 2^-11 for the weights'; values are below 127 * 0.021.
    assert ((o[at].double() - part[0].double()).abs() <= 2.0 ** -7 * part[0].double().abs() + 2.0 ** -10 * 2.7).all()
    live = ~part_lse[0].isinf() & ~lse[at].isinf()
    assert (lse[at] - part_lse[0])[live].abs().max() <= 2.0 ** -16 if live.any() else True


class _Only:
    """Sequence b of a cache without its first page."""

    def __init__(self, c, b):
        self.codes = c.codes
        self.gpu = (*c.gpu[:4], c.gpu[4][b:b + 1, 1:].contiguous())


@WIDTHS
def test_matches_decode_of_joined_histories(A, room):
    """A prefix that ends with a page: attn_decode_int8 over both parts in one table, within both roundings."""
    H, Hkv, d, page, n0, lens = 8, 2, 64, 16, 320, [5, 40, 100]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((3, 1, H, d), 1).cuda()
    o, lse = call(A, q, c, pre, n0, lens, room)
    width = 20 + c.gpu[4].shape[1]
    table = ints([(pre + t + [-1] * width)[:width] for t in c.tables])
    o2, lse2 = A.attn_decode_int8(q, *c.gpu[:4], table, ints([n0 + n for n in lens]))
    A.attn_check_status()
    # Both are within 2^-8 of a value for its rounding, and 2^-11 for the weights'; values are below 127 * 0.021.
    assert ((o.double() - o2.double()).abs() <= 2.0 ** -7 * o.double().abs() + 2.0 ** -10 * 2.7).all()
    assert (lse - lse2).abs().max() <= 2.0 ** -17


@WIDTHS
def test_views_bad_pages_and_lengths(A, room):
    """q as a view of a fused projection; a page out of range is not seen, lengths are cut, both are reported."""
    H, Hkv, d, page, n0, lens = 8, 2, 128, 32, 300, [70, 100, 20]
    c, pre = make(n0, lens, Hkv, page, d)
    qkv = normal((3, 2, H + 2 * Hkv, d), 2)
    q = qkv[:, :, :H]
    scale = 1 / math.sqrt(d)
    o, lse = call(A, qkv.cuda()[:, :, :H], c, pre, n0, lens, room)
    A.attn_check_status()
    check(c, pre, n0, q, lens, scale, o, lse)
    strided = q.transpose(0, 2).contiguous().cuda().transpose(0, 2)
    again = call(A, strided, c, pre, n0, lens, room)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    A.attn_check_status()
    for wrong in (-1, c.codes[0].shape[0], 2 ** 31 - 1):
        bad = list(pre)
        bad[4] = wrong
        o, lse = call(A, q.cuda(), c, bad, n0, lens, room)
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
        # As if that page were not in the prefix.
        check(c, pre[:4] + pre[5:], n0 - page, q, lens, scale, o, lse)
    o, lse = call(A, q.cuda(), c, pre, 10 ** 6, lens, room)
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    check(c, pre, len(pre) * page, q, lens, scale, o, lse)
    o, lse = call(A, q.cuda(), c, pre, -3, lens, room)
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    check(c, pre, 0, q, lens, scale, o, lse)
    for wrong in (10 ** 6, -3):
        o, lse = call(A, q.cuda(), c, pre, n0, [70, 100, wrong], room)
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
        check(c, pre, n0, q, lens, scale, o, lse, shown=(0, 1))
    A.attn_check_status()


@WIDTHS
def test_nan_rows_reach_no_other(A, room):
    H, Hkv, d, page, n0, lens = 16, 2, 64, 16, 400, [30, 7, 12] * 8
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((len(lens), 1, H, d), 1)
    good, good_lse = call(A, q.cuda(), c, pre, n0, lens, room)
    bad = q.clone()
    bad[5, 0, 3, 7] = torch.nan
    bad[9, 0, 8, 0] = torch.inf
    o, lse = call(A, bad.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    for b, h in ((5, 3), (9, 8)):
        assert o[b, 0, h].isnan().all() and lse[b, 0, h].isnan()
        o[b, 0, h], lse[b, 0, h] = good[b, 0, h], good_lse[b, 0, h]
    assert torch.equal(o, good) and torch.equal(lse, good_lse)


SPREAD = [(64, 1, 1), (128, 4, 1), (64, 4, 3), (128, 8, 9)]


@pytest.mark.parametrize("d,G,n_q", SPREAD)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n0", [300, 5000])
@WIDTHS
def test_value_scales_of_every_ratio(A, room, n0, page, d, G, n_q):
    """Value scales spread over 2^90 from page to page, one of them 0, and scores over some tens."""
    Hkv, lens = 2, [200, 90, 30]
    c, pre = make(n0, lens, Hkv, page, d)
    g = torch.Generator().manual_seed(n0 + page)
    c.scales[1] *= 2.0 ** torch.randint(-45, 46, c.scales[1].shape, generator=g)
    c.scales[1][pre[1]] = 0
    c.upload()
    q = normal((len(lens), n_q, Hkv * G, d), 1) * 2
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d,G,n_q", SPREAD)
@pytest.mark.parametrize("n0", [600, 4000])
@pytest.mark.parametrize("where", ["prefix", "own"])
@WIDTHS
def test_small_weights_of_large_values(A, room, where, n0, d, G, n_q):
    """The first 128 positions of the prefix, or all own ones, have weights of about 2^-118 of the row's largest and
    value scales 2^140 times the others': O is theirs."""
    Hkv, page, lens = 1, 32, [n_q + 60, n_q + 1]
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0][..., 0] = 0
    c.scales[0][:] = 0.002
    big = set(pre[:4]) if where == "prefix" else {p for t in c.tables for p in t}
    for p in range(len(c.codes[0])):
        c.scales[1][p] *= 2.0 ** (100 if p in big else -40)
        if p not in big:
            c.codes[0][p, ..., 0] = 100
    c.upload()
    q = normal((2, n_q, Hkv * G, d), 1)
    q[..., 0] = 592.0  # 100 * 0.002 * 592 = 118.4
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room, scale=math.log(2.0))
    A.attn_check_status()
    check(c, pre, n0, q, lens, math.log(2.0), o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("big", [40, 100])
@pytest.mark.parametrize("jump", [20.0, 100.0, 150.0])
@WIDTHS
def test_maximum_that_leaps(A, room, jump, big, d):
    """The score's maximum leaps where the value scale falls by 2^60 to 2^200, in both halves and tiles."""
    Hkv, page, n0, lens = 1, 32, 2000, [40, 40]
    for G in (2, 80):
        c, pre = make(n0, lens, Hkv, page, d)
        c.codes[0][..., 0] = 0
        c.scales[0][:] = 0.01
        for j, p in enumerate(pre):
            c.scales[1][p] *= 2.0 ** (big if j < 12 else -20 if big == 40 else -100)
            if j >= 12:
                c.codes[0][p, ..., 0] = 100
        c.upload()
        n_q = 1 if G == 2 else 2
        H = G if G <= 64 else 64
        q = normal((2, n_q, Hkv * H, d), 1)
        q[..., 0] = jump
        o, lse = call(A, q.cuda(), c, pre, n0, lens, room, scale=math.log(2.0))
        A.attn_check_status()
        assert o.isfinite().all()
        if jump < 126 or big == 40:  # else weights of p < 2^-126, which count as 0, would matter
            check(c, pre, n0, q, lens, math.log(2.0), o, lse)


@pytest.mark.parametrize("top", [2.0 ** 24 + 2, 2.0 ** 26, 2.0 ** 27 + 512, -(2.0 ** 25) - 100])
@pytest.mark.parametrize("d,G,n_q", [(64, 1, 1), (128, 4, 5), (64, 64, 3)])
@pytest.mark.parametrize("n0", [200, 9000])
@WIDTHS
def test_scores_beyond_the_exponent(A, room, n0, d, G, n_q, top):
    """The largest score in base 2 is `top`, where FP32 no longer holds whole numbers: one key of the own part and two of
    the prefix have it, far above all others, and the same value row, which is O exactly."""
    page, Hkv, lens = 32, 2, [n_q + 40, n_q]
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0][:] = 0
    c.codes[0][..., 0] = 60 if top > 0 else -127
    c.scales[0][:] = abs(top) / 100 * 2.0 ** -10
    c.scales[1][:] = 0.25
    row = torch.randint(-127, 128, (Hkv, d), generator=torch.Generator().manual_seed(1), dtype=torch.int8)
    for p, at in ((pre[0], 3), (pre[(n0 - 1) // page], (n0 - 1) % page), (c.tables[0][0], 0), (c.tables[1][0], 0)):
        c.codes[0][p, :, at, 0] = 100 if top > 0 else -100
        c.codes[1][p, :, at] = row
    c.upload()
    q = torch.zeros((2, n_q, Hkv * G, d), dtype=BF)
    q[..., 0] = 2.0 ** 10
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room, scale=math.log(2.0))
    A.attn_check_status()
    want = (row.double() * 0.25).repeat_interleave(G, 0)
    # The weights 1/3 of the parts sum to 1 within 2^-22, which O's rounding to BF16 (the row is a BF16 number) drops.
    assert (o.cpu().double() == want).all()
    # The roundings of test_decode_scores_beyond_the_exponent, and one of the factor's power of two more.
    assert ((lse.cpu().double() / (top * math.log(2.0)) - 1).abs() <= (10 + 1.6) * 2.0 ** -24 + 2.0 ** -40).all()


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 90])
@WIDTHS
def test_queries_of_extreme_size(A, room, size):
    """q and the keys' scales that only their products bring back into range."""
    H, Hkv, d, page, n0, lens = 8, 2, 64, 32, 500, [20, 60]
    c, pre = make(n0, lens, Hkv, page, d)
    c.scales[0] /= size
    c.upload()
    q = normal((2, 1, H, d), 1) * size
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@WIDTHS
def test_largest_values(A, room):
    """Values up to 2^127: no sum on the way overflows."""
    H, Hkv, d, page, n0, lens = 8, 2, 128, 32, 3000, [50, 3]
    c, pre = make(n0, lens, Hkv, page, d)
    c.scales[1][:] = 2.0 ** 120
    c.upload()
    q = normal((2, 1, H, d), 1)
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@WIDTHS
def test_the_same_call_twice_in_a_graph_and_on_two_streams(A, room):
    H, Hkv, d, page, n0 = 16, 2, 128, 64, 4000
    lens = [1 + 61 * b % 200 for b in range(20)]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((len(lens), 1, H, d), 1).cuda()
    first = call(A, q, c, pre, n0, lens, room)
    second = call(A, q, c, pre, n0, lens, room, scale=1 / math.sqrt(d))
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    table = pre + [-1] * (room // page)
    args = ints(table), ints([n0]), c.gpu[4], ints(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        third = A.attn_decode_shared_int8(q, *c.gpu[:4], *args, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, third))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(5):
                outs.append(A.attn_decode_shared_int8(q, *c.gpu[:4], *args))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for got in outs for x, y in zip(first, got))
    # Captured, then replayed on another prefix and other lengths.
    o, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])
    ws = torch.empty(1 + A.attn_decode_shared_int8_workspace_bytes(20, 1, H, Hkv, d, page, len(table), c.gpu[4].shape[1]),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        A.attn_decode_shared_int8(q, *c.gpu[:4], *args, o=o, lse=lse, workspace=ws)
    for n1, other in ((n0, lens), (77, lens[::-1]), (0, lens), (1500, [0] * 20)):
        other = [min(n, len(t) * page) for n, t in zip(other, c.tables)]
        args[1].copy_(ints([n1]))
        args[3].copy_(ints(other))
        ws.fill_(255)
        graph.replay()
        A.attn_check_status()
        check(c, pre, n1, q.cpu(), other, 1 / math.sqrt(d), o, lse, shown=(0, 3, 19))


@pytest.mark.parametrize("d,page", [(128, 128), (128, 16), (64, 64)])
@pytest.mark.parametrize("B,H,Hkv,n_q,n0,own", [(64, 32, 8, 1, 8000, 1), (64, 32, 8, 1, 8000, 100), (16, 32, 8, 1, 20000, 9),
                                               (100, 8, 2, 4, 3000, 4), (80, 8, 2, 16, 0, 2000), (80, 8, 2, 16, 0, 300)])
def test_same_bits_again_and_again(A, B, H, Hkv, n_q, n0, own, d, page):
    """Nothing that is read is overwritten early: many calls back to back, in both parts and every form of them, give the
    same bits."""
    lens = [own + (37 * b) % 100 if own > 200 else own for b in range(B)]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, n_q, H, d), 1).cuda()
    args = ints(pre + [-1] * (WIDE // page)), ints([n0]), c.gpu[4], ints(lens)
    first = A.attn_decode_shared_int8(q, *c.gpu[:4], *args)
    for _ in range(25):
        again = A.attn_decode_shared_int8(q, *c.gpu[:4], *args)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    A.attn_check_status()


def test_refusals(A):
    c, pre = make(40, [5], 2, 16, 64)
    q = normal((1, 1, 4, 64), 0).cuda()
    p, n, lens = ints(pre), ints([40]), ints([5])
    for args in ((q.half(), *c.gpu[:4], p, n, c.gpu[4], lens), (q, *c.gpu[:4], p.long(), n, c.gpu[4], lens),
                 (q, *c.gpu[:4], p[None], n, c.gpu[4], lens), (q, *c.gpu[:4], p, p[:2], c.gpu[4], lens),
                 (q, *c.gpu[:4], p, n, c.gpu[4], p[:2]), (q, *c.gpu[:4], p.cpu(), n, c.gpu[4], lens),
                 (q[0], *c.gpu[:4], p, n, c.gpu[4], lens)):
        with pytest.raises(ValueError):
            A.attn_decode_shared_int8(*args)
    with pytest.raises(A.AttnError, match="prefix_blocks"):
        A.attn_decode_shared_int8(q, *c.gpu[:4], p[:0], n, c.gpu[4], lens)
    with pytest.raises(A.AttnError, match="workspace"):
        A.attn_decode_shared_int8(q, *c.gpu[:4], ints(pre * 2000), n, c.gpu[4], lens, workspace=torch.empty(
            100, dtype=torch.uint8, device="cuda"))  # a table that wide is split
    with pytest.raises(A.AttnError, match="multiple of H_kv"):
        A.attn_decode_shared_int8(normal((1, 1, 5, 64), 0).cuda(), *c.gpu[:4], p, n, c.gpu[4], lens)
    A.attn_check_status()


def test_prefix_beyond_four_gib(A):
    """Pages whose bytes lie past 2^32."""
    Hkv, page, d, H = 8, 128, 128, 16
    pages = 2 ** 32 // (Hkv * page * d) + 40
    at = [pages - 1, pages - 3, 5, pages - 2, pages - 7]
    k_cache, v_cache = (torch.zeros((pages, Hkv, page, d), dtype=torch.int8, device="cuda") for _ in range(2))
    k_scale, v_scale = (torch.zeros((pages, Hkv), device="cuda") for _ in range(2))
    c = Cache(5, Hkv, page, d, [[3, 4]])  # the same five pages, small enough for the host
    for i, (codes, scale) in enumerate(((k_cache, k_scale), (v_cache, v_scale))):
        codes[at], scale[at] = c.codes[i].cuda(), c.scales[i].cuda()
    q = normal((1, 1, H, d), 3)
    o, lse = A.attn_decode_shared_int8(q.cuda(), k_cache, v_cache, k_scale, v_scale, ints(at[:3]), ints([300]),
                                       ints([at[3:]]), ints([200]))
    A.attn_check_status()
    check(c, [0, 1, 2], 300, q, [200], 1 / math.sqrt(d), o, lse)


def test_steps_behind_a_prefix(A):
    """A serving run in one captured step: pages are reserved on the GPU, the step's rows appended, and attended over
    behind a shared prompt; drafts that are rejected give their pages back; a request ends and another begins."""
    H, Hkv, d, page, n_q, B, n0, width = 8, 2, 64, 16, 3, 4, 100, 6
    pages = 40
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
    pre, free = order[:-(-n0 // page)], order[-(-n0 // page):]
    c = Cache(pages, Hkv, page, d, [[] for _ in range(B)], width=width)
    table, stack, n_free = c.gpu[4], ints(free + [-1] * (pages - len(free))), ints([len(free)])
    books = [[-1] * width for _ in range(B)], list(free) + [-1] * (pages - len(free)), len(free)
    rows = torch.zeros((B, n_q, H + 2 * Hkv, d), dtype=BF, device="cuda")
    T = B * n_q
    held, wanted = ints([0] * B), ints([0] * B)
    lens, cu = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots, positions = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    o, lse = torch.zeros((B, n_q, H, d), dtype=BF, device="cuda"), torch.zeros((B, n_q, H), device="cuda")
    ws = torch.empty(1 + A.attn_decode_shared_int8_workspace_bytes(B, n_q, H, Hkv, d, page, len(pre), width),
                     dtype=torch.uint8, device="cuda")
    prefix, prefix_len = ints(pre), ints([n0])

    def step():
        A.attn_cache_reserve(table, held, wanted, stack, n_free, page, T, lens=lens, cu_seqlens=cu, slots=slots,
                             positions=positions)
        flat = rows.view(T, H + 2 * Hkv, d)
        A.attn_cache_append_int8(flat[:, H:H + Hkv], flat[:, H + Hkv:], *c.gpu, cu, held)
        A.attn_decode_shared_int8(rows[:, :, :H], *c.gpu[:4], prefix, prefix_len, table, lens, o=o, lse=lse, workspace=ws)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    have = [0] * B
    table_list, stack_list, free_count = books
    for s in range(14):
        x = normal((B, n_q, H + 2 * Hkv, d), 20 + s)
        rows.copy_(x)
        want = [n + n_q for n in have]
        held.copy_(ints(have))
        wanted.copy_(ints(want))
        graph.replay()
        A.attn_check_status()
        got = ref.reserve(table_list, have, want, stack_list, free_count, page, T, pages)
        free_count = got[4]
        assert got[0] == want  # pages suffice
        assert [y.tolist() for y in (lens, cu, slots, positions)] == list(got[:4])
        assert table.tolist() == table_list and n_free.item() == free_count
        c.tables = [[p for p in t if p >= 0] for t in table_list]
        flat = x.view(T, H + 2 * Hkv, d)
        c.append([flat[:, H:H + Hkv], flat[:, H + Hkv:]], got[1], have)
        assert c.equal()
        for t, slot in enumerate(slots.tolist()):  # where the rows lie
            codes = c.codes[0][slot // page, :, slot % page].double() * c.scales[0][slot // page].double()[:, None]
            assert (codes - flat[t, H:H + Hkv].double()).abs().max() <= 0.51 * c.scales[0][slot // page].max() + 1e-9
        check(c, pre, n0, x[:, :, :H], want, 1 / math.sqrt(d), o, lse)
        # One to three of the drafts are kept; a request ends when it has no room for more.
        have = [n + 1 + (s + b) % 3 for b, n in enumerate(have)]
        have = [0 if n + n_q > width * page or (s == 6 and b == 1) else n for b, n in enumerate(have)]
        A.attn_cache_reserve(table, lens, ints(have), stack, n_free, page, 0)
        got = ref.reserve(table_list, want, have, stack_list, free_count, page, 0, pages)
        free_count = got[4]
        assert table.tolist() == table_list and stack.tolist()[:free_count] == stack_list[:free_count]
    A.attn_check_status()
