"""Attention over a shared prefix: what must hold for either way of reading it, each with the way that it takes."""
import math

import pytest

from test_serving_gpu import A, Cache, ints, normal  # noqa: F401
from test_shared_gpu import WIDE, call, check, make
from test_shared_scales_gpu import by_units

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
# (Sequences, room in the prefix's table): read once for 256 rows of the tests here, or once a sequence.
BY = pytest.mark.parametrize("units,B,room", [(True, 8, WIDE), (False, 2, 0)])


def attend(A, units, q, c, pre, n0, lens, room, **kw):  # noqa: N803
    page, Hkv = c.codes[0].shape[2], c.codes[0].shape[1]
    assert by_units(A, q, Hkv, page, len(pre) + room // page, c.gpu[4].shape[1]) == units
    out = call(A, q.cuda(), c, pre, n0, lens, room, **kw)
    A.attn_check_status()
    return out


@BY
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("n_q", [1, 3])
def test_few_rows(A, units, B, room, n_q, G, d):
    Hkv, page, n0, lens = 2, 32, 700, [n_q + 5 * b for b in range(B)]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, n_q, Hkv * G, d), 1)
    o, lse = attend(A, units, q, c, pre, n0, lens, room)
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@BY
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 90])
def test_queries_of_extreme_size(A, units, B, room, size, d):
    """q and the keys' scales that only their products bring back into range."""
    H, Hkv, page, n0, lens = 8, 2, 32, 500, [20 + 9 * b for b in range(B)]
    c, pre = make(n0, lens, Hkv, page, d)
    c.scales[0] /= size
    c.upload()
    q = normal((B, 1, H, d), 1) * size
    o, lse = attend(A, units, q, c, pre, n0, lens, room)
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse)


@BY
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("big", [40, 100])
@pytest.mark.parametrize("jump", [20.0, 100.0, 124.0, 150.0])
@pytest.mark.parametrize("G", [1, 16])
def test_maximum_that_leaps(A, units, B, room, G, jump, big, d):
    """The score's maximum leaps where the value scale falls by 2^60 to 2^200, also by more than FP32's exponents: what
    then counts as 0 is within check's bound, which has those weights' own size."""
    Hkv, page, n0, lens = 1, 32, 2000, [40] * B
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0][..., 0] = 0
    c.scales[0][:] = 0.01
    for j, p in enumerate(pre):
        c.scales[1][p] *= 2.0 ** (big if j < 12 else -20 if big == 40 else -100)
        if j >= 12:
            c.codes[0][p, ..., 0] = 100
    c.upload()
    q = normal((B, 1, G, d), 1)
    q[..., 0] = jump
    o, lse = attend(A, units, q, c, pre, n0, lens, room, scale=math.log(2.0))
    assert o.isfinite().all()
    check(c, pre, n0, q, lens, math.log(2.0), o, lse)


@BY
@pytest.mark.parametrize("top", [2.0 ** 24 + 2, 2.0 ** 26, 2.0 ** 27 + 512, -(2.0 ** 25) - 100])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_beyond_the_exponent(A, units, B, room, d, top):
    """As its namesake in test_shared_gpu, at one row a sequence: the keys of the largest score have the same value row."""
    page, Hkv, n0, n_q, G = 32, 2, 9000 if units else 200, 1, 1
    lens = [n_q + 40] * (B - 1) + [n_q]
    c, pre = make(n0, lens, Hkv, page, d)
    c.codes[0][:] = 0
    c.codes[0][..., 0] = 60 if top > 0 else -127
    c.scales[0][:] = abs(top) / 100 * 2.0 ** -10
    c.scales[1][:] = 0.25
    row = torch.randint(-127, 128, (Hkv, d), generator=torch.Generator().manual_seed(1), dtype=torch.int8)
    for p, at in ((pre[0], 3), (pre[(n0 - 1) // page], (n0 - 1) % page), *((t[0], 0) for t in c.tables)):
        c.codes[0][p, :, at, 0] = 100 if top > 0 else -100
        c.codes[1][p, :, at] = row
    c.upload()
    q = torch.zeros((B, n_q, Hkv * G, d), dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** 10
    o, lse = attend(A, units, q, c, pre, n0, lens, room, scale=math.log(2.0))
    want = (row.double() * 0.25).repeat_interleave(G, 0)
    # The weights 1/3 of the parts sum to 1 within 2^-22, which O's rounding to BF16 (the row is a BF16 number) drops.
    assert (o.cpu().double() == want).all()
    # The scores' own roundings, and that of the factor's power of two, as in the namesake.
    assert ((lse.cpu().double() / (top * math.log(2.0)) - 1).abs() <= (10 + 1.6) * 2.0 ** -24 + 2.0 ** -40).all()


@BY
def test_without_the_tensor_binding(A, units, B, room, monkeypatch):
    from precision_numerics_gb300 import attn

    lens = [9 + 17 * b for b in range(B)]
    c, pre = make(300, lens, 2, 16, 64)
    q = normal((B, 1, 8, 64), 1)
    want = attend(A, units, q, c, pre, 300, lens, room)
    monkeypatch.setattr(attn, "_BINDING", attn._NoBinding)
    got = attend(A, units, q, c, pre, 300, lens, room)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    attend(A, units, q, c, pre, 300, lens, room, o=o, lse=lse)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_pages_beyond_four_gib(A):
    """Pages whose bytes lie past 2^32, of the prefix read once for 256 rows (of one row tile and of two), and of own
    positions by units."""
    Hkv, page, d = 8, 128, 128
    pages = 2 ** 32 // (Hkv * page * d) + 40
    at = [pages - 1, pages - 3, 5, pages - 2, pages - 7]
    k_cache, v_cache = (torch.zeros((pages, Hkv, page, d), dtype=torch.int8, device="cuda") for _ in range(2))
    k_scale, v_scale = (torch.zeros((pages, Hkv), device="cuda") for _ in range(2))
    for B, G, n_q in ((8, 2, 1), (64, 4, 1), (20, 2, 20)):
        c = Cache(5, Hkv, page, d, [[3, 4]] * B)  # the same five pages, small enough for the host
        for i, (codes, scale) in enumerate(((k_cache, k_scale), (v_cache, v_scale))):
            codes[at], scale[at] = c.codes[i].cuda(), c.scales[i].cuda()
        q, lens = normal((B, n_q, Hkv * G, d), 3), [200 + b % 50 for b in range(B)]
        blocks = WIDE // page
        assert by_units(A, q, Hkv, page, blocks, 2)
        o, lse = A.attn_decode_shared_int8(q.cuda(), k_cache, v_cache, k_scale, v_scale, ints(at[:3] + [-1] * (blocks - 3)),
                                           ints([300]), ints([at[3:]] * B), ints(lens))
        A.attn_check_status()
        check(c, [0, 1, 2], 300, q, lens, 1 / math.sqrt(d), o, lse, shown=(0, 1, B - 1))
