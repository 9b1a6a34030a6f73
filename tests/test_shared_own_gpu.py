"""Attention over a shared prefix with many new tokens: which kernel has the own positions follows from the room that
the table has for them."""
import math

import pytest

from test_serving_gpu import A, ints, normal  # noqa: F401
from test_shared_gpu import call, check, make

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n_q", [(4, 15), (4, 16), (8, 17), (8, 32)])
@pytest.mark.parametrize("beyond", [0, 1])
def test_both_sides_of_the_room(A, beyond, G, n_q, d):
    """Histories of up to rows^2 / 8 positions, in a table with no more room than that and with a page more; 60 rows a
    sequence and key head, 64, 136 and 256, from which on the room does not count; the same bits again and again."""
    B, Hkv, page, n0 = 80, 2, 32, 500
    room = min((G * n_q) ** 2 // 8, 3000) // page * page
    lens = [room, 0, 1, n_q] + [n_q + (b * b * 131) % (room - n_q) for b in range(B - 4)]
    c, pre = make(n0, lens, Hkv, page, d, width=room // page + beyond)
    q = normal((B, n_q, Hkv * G, d), 1)
    args = q.cuda(), *c.gpu[:4], ints(pre), ints([n0]), c.gpu[4], ints(lens)
    o, lse = A.attn_decode_shared_int8(*args)
    A.attn_check_status()
    check(c, pre, n0, q, lens, 1 / math.sqrt(d), o, lse, shown=(0, 1, 2, 3, B - 1))
    for _ in range(10):
        again = A.attn_decode_shared_int8(*args)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    A.attn_check_status()


def test_one_long_history_is_not_one_block(A):
    """A history of 100000 positions among 19 short ones takes no more than a few times what attn_decode_int8, which deals
    it to all SMs, needs for the own positions alone (it took 9 times that with a block a key head)."""
    B, H, Hkv, d, page, n_q, n0 = 20, 32, 8, 128, 64, 16, 200
    lens = [100000] + [100 + 7 * b for b in range(B - 1)]
    c, pre = make(n0, lens, Hkv, page, d)
    q = normal((B, n_q, H, d), 1).cuda()

    def us(f, times=10):
        for _ in range(3):
            f()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(times):
            f()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) / times * 1000

    pre_table, n, own = ints(pre), ints([n0]), ints(lens)
    alone = us(lambda: A.attn_decode_int8(q, *c.gpu, own))
    both = us(lambda: A.attn_decode_shared_int8(q, *c.gpu[:4], pre_table, n, c.gpu[4], own))
    A.attn_check_status()
    print(f"own positions {alone:.0f} us, behind a prefix {both:.0f} us")
    assert both < 2.5 * alone
    o, lse = call(A, q, c, pre, n0, lens)
    check(c, pre, n0, q.cpu(), lens, 1 / math.sqrt(d), o, lse, shown=(1, B - 1))
