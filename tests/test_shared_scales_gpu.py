"""Attention over a shared prefix: value scales far apart, in every order of the pages and in each of its kernels."""
import math

import pytest

from test_serving_gpu import A, Cache, normal, scattered  # noqa: F401
from test_shared_gpu import WIDE, call, check, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def by_units(A, q, Hkv, page, blocks, max_blocks):  # noqa: N803
    """Whether the prefix is read once for 256 rows: only then the workspace has room for a part of 256 rows for each of
    the runs, of which there are as many as SMs."""
    B, n_q, H, d = q.shape
    return A.attn_decode_shared_int8_workspace_bytes(B, n_q, H, Hkv, d, page, blocks, max_blocks) > 128 * 256 * (d + 2) * 4


# Where the two kinds of pages lie: in the prefix, read once for 256 rows (by units of two row tiles, and of one, whose
# key tiles two halves take by turns) or once a sequence, or among the own positions of many new tokens, by units.
# (B, Hkv, G, n_q, how often the pattern comes: runs have several key tiles)
FORMS = {"two": (64, 8, 8, 1, 8), "one": (32, 8, 4, 1, 24), "by sequence": (2, 2, 2, 2, 1), "own": (80, 2, 8, 16, 1)}
GAPS = [(100, 118), (112, 123), (112, 132), (118, 121), (118, 123), (118, 126), (118, 140), (124, 123), (124, 129),
        (125, 130)]
PLACES = [(1, 512), (128, 512), (33, 490), (130, 510), (7, 383)]
CASES = [(form, *place, *gap, d) for form in FORMS for place in (PLACES[1:3] if form == "one" else PLACES) for gap in GAPS
         for d in (64, 128) if gap in GAPS[4::4] or d == 128 and form != "one"]


@pytest.mark.parametrize("form,count,first,gap,ratio,d", CASES)
def test_large_values_of_small_weights_last(A, form, count, first, gap, ratio, d):
    """The pages from position `first` on, `count` positions, have weights of 2^-gap of the row's largest and value scales
    2^ratio times those before them, so that what they add to O is 2^(ratio - gap) of the others': in the key tile of the
    others, and in one of their own behind theirs."""
    B, Hkv, G, n_q, times = FORMS[form]
    page, n = 16, first + count
    pages = -(-n // page)
    n = n if times == 1 else pages * page * times
    lens = [n - b % 3 for b in range(B)] if form == "own" else [1 + b % 3 for b in range(B)]
    n0 = 40 if form == "own" else n
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0].remainder_(9).sub_(4)  # scores stay within some tenths of what channel 0 makes them
    c.codes[0][..., 0] = 100
    c.scales[0][:] = 0.002
    c.scales[1] *= 2.0 ** -40
    for table in c.tables if form == "own" else [pre]:
        last = [p for j, p in enumerate(table) if (j % pages + 1) * page > first]
        c.scales[1][last] *= 2.0 ** (ratio // 2)  # (in two steps: 2^128 is no FP32 number)
        c.scales[1][last] *= 2.0 ** (ratio - ratio // 2)
        c.codes[0][last, ..., 0] = 0
    c.upload()
    q = normal((B, n_q, Hkv * G, d), 1)
    q[..., 0] = gap / 0.2  # 100 * 0.002 * gap / 0.2 = gap
    room = 0 if form == "by sequence" else WIDE
    assert by_units(A, q, Hkv, page, len(pre) + room // page, c.gpu[4].shape[1]) == (form != "by sequence")
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room, scale=math.log(2.0))
    A.attn_check_status()
    check(c, pre, n0, q, lens, math.log(2.0), o, lse, shown=(0, 1, B - 1))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 32), (64, 64)])
@pytest.mark.parametrize("n", [5, 130, 300, 517])
@pytest.mark.parametrize("absent", [False, True])
def test_scales_of_pages_in_no_table_decide_nothing(A, form, absent, n, page, d):
    """Pages that no table names, page 0 among them, hold any scales at all (they may never have been written, or another
    stream writes them): the last key tile ends inside, and `absent` pages are out of range.  The value scales grow from
    page to page, so that a row's references have to move in the last tile as well."""
    B, Hkv, G, n_q, _ = FORMS[form]
    lens = [n + b % 3 for b in range(B)] if form == "own" else [1 + b % 3 for b in range(B)]
    n0 = 40 if form == "own" else n
    tables, pages = scattered([-(-n0 // page)] + [-(-x // page) for x in lens], 7)
    tables = [[p + 1 for p in t] for t in tables]
    c = Cache(pages + 1, Hkv, page, d, tables[1:])
    for table in tables:
        for j, p in enumerate(table):
            c.scales[1][p] *= 2.0 ** (3 * j)
    used = [p for t in tables for p in t]
    rest = [p for p in range(pages + 1) if p not in set(used)]
    assert 0 in rest
    pre = list(tables[0])
    if absent:
        (pre if form != "own" else c.tables[0])[n // page // 2] = pages + 1
        c = Cache(pages + 1, Hkv, page, d, c.tables) if form == "own" else c
    q = normal((B, n_q, Hkv * G, d), 1).cuda()
    room, want = 0 if form == "by sequence" else WIDE, None
    assert by_units(A, q, Hkv, page, len(pre) + room // page, c.gpu[4].shape[1]) == (form != "by sequence")
    for poison in (0.01, 0.0, -1.0, 2.0 ** 100, torch.inf, -torch.inf, torch.nan):
        for scales in c.scales:
            scales[rest] = poison
        c.upload()
        got = call(A, q, c, pre, n0, lens, room)
        if absent:
            with pytest.raises(A.AttnError, match="out of range"):
                A.attn_check_status()
        A.attn_check_status()
        want = want or got
        assert got[0].isfinite().all() and all(torch.equal(x, y) for x, y in zip(want, got)), poison


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [120.0, 126.9, 127.9])
def test_value_scales_next_to_the_last(A, form, d, size):
    """Value scales up to FP32's end whose codes are small enough for finite values: +-1 at 2^127.9, +-100 at 2^120."""
    B, Hkv, G, n_q, times = FORMS[form]
    page, n = 16, 300 * times
    lens = [n - b % 3 for b in range(B)] if form == "own" else [1 + b % 3 for b in range(B)]
    n0 = 40 if form == "own" else n
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[1].remainder_(3).sub_(1)
    if size == 120.0:
        c.codes[1].mul_(100)
    c.scales[1][:] = 2.0 ** size
    c.upload()
    q = normal((B, n_q, Hkv * G, d), 1)
    room = 0 if form == "by sequence" else WIDE
    assert by_units(A, q, Hkv, page, len(pre) + room // page, c.gpu[4].shape[1]) == (form != "by sequence")
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room)
    A.attn_check_status()
    assert o.isfinite().all()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse, shown=(0, 1, B - 1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["two", "one"])
def test_parts_whose_maximum_lags(A, form, d):
    """In the first half of the prefix key tiles of score 0 and of score 31 take turns, with value scales that fall as
    much but for 2^3, so that a part's reference stays where the first tile left it; the second half has score 155 and value
    scales 2^124 smaller, so that both halves weigh alike in O.  Weights of 2^-124 are kept."""
    B, Hkv, G, n_q, times = FORMS[form]
    page, tiles = 16, 8 * times
    n0, lens = 128 * tiles, [1 + b % 3 for b in range(B)]
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0].remainder_(9).sub_(4)
    c.codes[0][..., 0] = 0
    c.scales[0][:] = 0.002
    c.scales[1].fill_(2.0 ** 60)
    for table in c.tables:  # own positions have a weight of 2^-155 and next to no value
        c.scales[1][table] = 2.0 ** -100
    for j, p in enumerate(pre):
        tile = j // 8
        if tile >= tiles // 2:
            c.codes[0][p, ..., 0] = 100
            c.scales[1][p] *= 2.0 ** -124
        elif tile % 2:
            c.codes[1][p] = 100 if j % 8 == 3 else 0
            if j % 8 == 3:
                c.codes[0][p, ..., 0] = 20
        else:
            c.codes[1][p] = 1 if j % 8 == 2 else 0  # what the weights of 2^-155 are worth stays small
            if j % 8 == 2:
                c.scales[1][p] *= 2.0 ** 28
    c.upload()
    q = normal((B, n_q, Hkv * G, d), 1)
    q[..., 0] = 776.0  # 100 * 0.002 * 776 = 155.2
    assert by_units(A, q, Hkv, page, len(pre) + WIDE // page, c.gpu[4].shape[1])
    o, lse = call(A, q.cuda(), c, pre, n0, lens, WIDE, scale=math.log(2.0))
    A.attn_check_status()
    check(c, pre, n0, q, lens, math.log(2.0), o, lse, shown=(0, 1, B - 1))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("course", ["rise", "cancel", "turns"])
@pytest.mark.parametrize("gap,span,run,d", [(124, 110, 16, 64), (124, 110, 8, 128), (60, 60, 2, 128), (30, 20, 9, 64)])
def test_scores_and_value_scales_of_opposite_course(A, form, course, gap, span, run, d):
    """Scores rise by `gap` in base 2 over the positions, `run` pages at a time, while value scales fall by 2^(2 span), or
    by as much as the scores rise, or both change by turns: the largest weights of the values lie anywhere in the row, at
    any distance from its largest score, and references lag behind the scores."""
    B, Hkv, G, n_q, times = FORMS[form]
    page, n = 16, 407 * times
    lens = [n - b % 3 for b in range(B)] if form == "own" else [1 + b % 3 for b in range(B)]
    n0 = 40 if form == "own" else n
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0].remainder_(9).sub_(4)
    c.scales[0][:] = 0.002
    for table in c.tables if form == "own" else [pre]:
        for j, p in enumerate(table):
            x = j // run % 2 if course == "turns" else j // run / max(1, (len(table) - 1) // run)
            c.codes[0][p, ..., 0] = round(100 * x)
            e = gap / 2 - gap * x if course == "cancel" else span - 2 * span * x
            c.scales[1][p] *= 2.0 ** e
    c.upload()
    q = normal((B, n_q, Hkv * G, d), 1)
    q[..., 0] = gap / 0.2
    room = 0 if form == "by sequence" else WIDE
    assert by_units(A, q, Hkv, page, len(pre) + room // page, c.gpu[4].shape[1]) == (form != "by sequence")
    o, lse = call(A, q.cuda(), c, pre, n0, lens, room, scale=math.log(2.0))
    A.attn_check_status()
    check(c, pre, n0, q, lens, math.log(2.0), o, lse, shown=(0, B - 1))
