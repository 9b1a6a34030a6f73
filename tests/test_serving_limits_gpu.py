"""Serving operators at the ends of their ranges."""
import math

import pytest

import serving_ref as ref
from test_serving_gpu import A, BF, Cache, ints, scattered  # noqa: F401

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
