"""Attention over a shared prefix read once for 256 rows: joins of many parts a row."""
import math

import pytest

from test_serving_gpu import A, normal  # noqa: F401
from test_shared_gpu import WIDE, call, check, make
from test_shared_scales_gpu import by_units

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,n0", [(64, 8, 1, 100000), (32, 8, 1, 100001), (16, 8, 1, 99999), (6, 5, 1, 100000),
                                        (40, 7, 1, 90000), (9, 16, 2, 45000)])
def test_joins_of_many_parts(A, B, H, Hkv, n0, d):
    """More parts a row than the join holds the shares of (64): one unit of two row tiles, or of one, whose halves leave
    a part each, two units, and one of each kind."""
    page, lens = 64, [1 + 37 * b % 90 for b in range(B)]
    rows, runs = B * H // Hkv, torch.cuda.get_device_properties(0).multi_processor_count
    units, halves = -(-rows // 256) * Hkv, 2 if rows <= 128 else 1
    assert -(-n0 // 128) >= 2 * runs and runs // units * halves > 64  # of a run's two key tiles at least
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, 1, H, d), 1)
    assert by_units(A, q, Hkv, page, len(pre), c.gpu[4].shape[1])
    o, lse = call(A, q.cuda(), c, pre, n0, lens)
    A.attn_check_status()
    scale = 1 / math.sqrt(d)
    check(c, pre, n0, q, lens, scale, o, lse, shown=(0, B // 2, B - 1))
    # A weight that only one of the parts has: the last position of the prefix is the largest key by far.
    for n1, room in ((n0 - 1, 0), (65 * 256 + 1, WIDE)):
        c.codes[0][pre[n1 // page], :, n1 % page] = 127
        c.scales[0][pre[n1 // page]] = 0.2
        c.upload()
        o, lse = call(A, q.abs().cuda(), c, pre, n1 + 1, lens, room)
        A.attn_check_status()
        check(c, pre, n1 + 1, q.abs(), lens, scale, o, lse, shown=(0, B - 1))
    again = call(A, q.abs().cuda(), c, pre, n1 + 1, lens, room)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
