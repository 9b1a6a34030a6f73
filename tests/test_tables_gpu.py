"""Block tables, offsets and slots built on the GPU, against lists."""
import random

import pytest

import serving_ref as ref
from test_serving_gpu import A, ints  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Books:
    """Table and stack, here and on the GPU."""

    def __init__(self, held, page, width, free, seed=0, spare=0):
        self.page, rng = page, random.Random(seed)
        up = [-(-n // page) for n in held]
        self.pages = sum(up) + free + spare
        order = list(range(self.pages))
        rng.shuffle(order)
        at, self.table = 0, []
        for n in up:
            self.table.append(order[at:at + n] + [-1] * (width - n))
            at += n
        self.stack = order[at:at + free] + [-1] * (self.pages - free)
        self.free = free
        self.gpu = ints(self.table), ints(self.stack), ints([free])

    def step(self, A, held, wanted, T, **outs):  # noqa: N803
        want = ref.reserve(self.table, held, wanted, self.stack, self.free, self.page, T, self.pages)
        self.free = want[4]
        table, stack, free = self.gpu
        got = A.attn_cache_reserve(table, ints(held), ints(wanted), stack, free, self.page, T, **outs)
        for name, g, w in zip(("lens", "cu_seqlens", "slots", "positions"), got, want):
            assert g.tolist() == w, name
        assert table.tolist() == self.table
        assert stack.tolist() == self.stack and free.item() == self.free
        return got


def lengths(n, most, seed, ends=0.2):
    rng = random.Random(seed)
    held = [rng.choice([0, rng.randint(0, most)]) for _ in range(n)]
    wanted = [0 if rng.random() < ends else rng.randint(0, most) if rng.random() < 0.2 else min(most, h + rng.randint(0, 40))
              for h in held]
    return held, wanted


def new_tokens(held, wanted):
    return sum(max(0, w - h) for h, w in zip(held, wanted))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 500, 1023, 1024, 1025, 3000])
def test_steps(A, n, page):
    """Steps of many kinds one after the other, each then taken back and done again."""
    most = 300
    held, wanted = lengths(n, most, n + page)
    books = Books(held, page, -(-most // page) + 1, free=n, seed=n)
    start = [list(r) for r in books.table], books.free
    lens = books.step(A, held, wanted, new_tokens(held, wanted))[0].tolist()
    books.step(A, lens, held, new_tokens(lens, held) + 3)
    assert (books.table, books.free) == start
    books.step(A, held, wanted, new_tokens(held, wanted) + 1)
    for i in range(3):
        _, wanted = lengths(n, most, i)
        lens = books.step(A, lens, wanted, new_tokens(lens, wanted))[0].tolist()
    A.attn_check_status()


@pytest.mark.parametrize("n,T", [(1, 1), (3, 5000), (40, 70000), (600, 70001), (2000, 300000)])
def test_many_tokens(A, n, T):
    """Slots by one CTA, a cluster and the second kernel; sequences of nothing among long ones."""
    rng, page = random.Random(n), 16
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    new = [b - a for a, b in zip([0, *cuts], [*cuts, T])]
    held = [rng.randint(0, 50) for _ in new]
    wanted = [h + x for h, x in zip(held, new)]
    width = -(-max(wanted) // page)
    books = Books(held, page, width, free=sum(-(-w // page) for w in wanted), seed=n)
    lens = books.step(A, held, wanted, T)[0].tolist()
    books.step(A, lens, [0] * n, 0)  # everything ends, T = 0
    A.attn_check_status()


def test_many_sequences_without_tokens(A):
    """Slots of many tokens where thousands of sequences between them have none."""
    page, n = 16, 9000
    held = [3] * n
    wanted = [3 + (20000 if b in (2, 4100, 8999) else 1 if b % 3000 == 7 else 0) for b in range(n)]
    T = new_tokens(held, wanted) + 77
    books = Books(held, page, -(-20003 // page), free=3 * 1260, seed=3)
    lens = books.step(A, held, wanted, T)[0].tolist()
    books.step(A, lens, held, 1)
    A.attn_check_status()


@pytest.mark.parametrize("free", [0, 1, 7, 30, 31, 60])
def test_scarce_pages(A, free):
    """Requests are served in order as long as pages last; what ends in the same step counts in."""
    held = [0, 40, 16, 3, 100, 0, 64]
    wanted = [33, 0, 17, 6, 300, 1, 80]
    books = Books(held, 16, 20, free)
    lens = books.step(A, held, wanted, new_tokens(held, wanted))[0].tolist()
    books.step(A, lens, held, 200)
    A.attn_check_status()


def test_lengths_out_of_range(A):
    """Such a sequence is left as it is and reported; the others are served."""
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        for held, wanted in (([5, bad, 20], [40, 3, 0]), ([5, 20, 20], [40, bad, 0])):
            books = Books([5, 20, 20], 16, 4, free=9)
            books.step(A, held, wanted, 40)
            with pytest.raises(A.AttnError, match="tables [1-9]"):
                A.attn_check_status()
    A.attn_check_status()


def test_bad_numbers(A):
    """Pages out of range in the table or on the stack become -1, a stack that is too full drops pages, a count
    out of range is cut, and more tokens than T are left out; all reported."""
    def books():
        return Books([20, 20], 16, 4, free=3, spare=2)

    b = books()
    b.table[0][1] = b.pages
    b.gpu[0][0, 1] = b.pages
    b.step(A, [20, 20], [3, 40], 20)  # given back, and taken by the second
    with pytest.raises(A.AttnError, match="tables"):
        A.attn_check_status()
    b = books()
    b.stack[2] = -7
    b.gpu[1][2] = -7
    b.step(A, [20, 20], [20, 50], 30)
    with pytest.raises(A.AttnError, match="tables"):
        A.attn_check_status()
    b = books()
    b.free = b.pages - 1
    b.stack[3:5] = [0, 0]
    b.gpu[1][3:5] = 0
    b.gpu[2].fill_(b.free)
    b.step(A, [20, 20], [0, 0], 0)
    assert b.free == b.pages
    with pytest.raises(A.AttnError, match="tables"):
        A.attn_check_status()
    for wrong in (-5, 10 ** 6):
        b = books()
        b.free = wrong
        b.gpu[2].fill_(wrong)
        b.step(A, [20, 20], [33, 20], 13)
        with pytest.raises(A.AttnError, match="tables"):
            A.attn_check_status()
    b = books()
    b.table[0][1] = -1  # the page that is begun
    b.gpu[0][0, 1] = -1
    b.step(A, [20, 20], [25, 20], 5)
    with pytest.raises(A.AttnError, match="tables"):
        A.attn_check_status()
    b = books()
    b.step(A, [20, 20], [33, 40], 17)
    with pytest.raises(A.AttnError, match="tables"):
        A.attn_check_status()
    A.attn_check_status()


def test_outputs_streams_and_refusals(A):
    """Outputs that are passed in, views of one buffer at odd places; a stream; what overlaps or has another type."""
    held, wanted = [20, 5, 0], [50, 0, 17]
    T = new_tokens(held, wanted)
    buf = torch.full((3 + 4 + 2 * T + 7,), 99, dtype=torch.int32, device="cuda")
    outs = dict(lens=buf[1:4], cu_seqlens=buf[4:8], slots=buf[9:9 + T], positions=buf[9 + T:9 + 2 * T])
    Books(held, 16, 5, free=9).step(A, held, wanted, T, **outs)
    assert buf[0] == 99 and buf[8] == 99 and (buf[9 + 2 * T:] == 99).all()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        b = Books(held, 16, 5, free=9)
        torch.cuda.synchronize()
        want = ref.reserve(b.table, held, wanted, b.stack, b.free, 16, T, b.pages)
        args = ints(held), ints(wanted)
        torch.cuda.synchronize()
        got = A.attn_cache_reserve(b.gpu[0], *args, *b.gpu[1:], 16, T, stream=stream)
        A.attn_check_status(side)
        torch.cuda.synchronize()
        assert [g.tolist() for g in got] == list(want[:4])
    table, stack, free = Books(held, 16, 5, free=9).gpu
    h, w = ints(held), ints(wanted)
    for bad in (dict(lens=h), dict(lens=w), dict(cu_seqlens=stack[:4]), dict(slots=table.view(-1)[:4], T=4),
                dict(slots=buf[:4], positions=buf[3:7], T=4)):
        n = bad.pop("T", T)
        with pytest.raises(A.AttnError, match="overlap"):
            A.attn_cache_reserve(table, h, w, stack, free, 16, n, **bad)
    with pytest.raises(A.AttnError, match="overlap"):
        A.attn_cache_reserve(table, h, w, stack, w[:1], 16, T)
    for args in ((table.long(), h, w, stack, free), (table, h[:2], w, stack, free), (table, h, w.long(), stack, free),
                 (table, h, w, stack, stack[:2]), (table.t(), h, w, stack, free)):
        with pytest.raises(ValueError):
            A.attn_cache_reserve(*args, 16, T)
    with pytest.raises(A.AttnError, match="page_size"):
        A.attn_cache_reserve(table, h, w, stack, free, 48, T)
    with pytest.raises((A.AttnError, RuntimeError, ValueError)):
        A.attn_cache_reserve(table, h, w, stack, free, 16, -1)
    A.attn_check_status()


def test_in_a_graph(A):
    """A captured step replayed on new lengths, with its outputs in place."""
    held, wanted = [0, 30, 7], [9, 31, 40]
    T = 60
    b = Books(held, 16, 5, free=12, seed=3)
    h, w = ints(held), ints(wanted)
    outs = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (3, 4, T, T)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        A.attn_cache_reserve(b.gpu[0], h, w, *b.gpu[1:], 16, T, lens=outs[0], cu_seqlens=outs[1], slots=outs[2],
                             positions=outs[3])
    reported = 0
    for _ in range(4):
        h.copy_(ints(held))
        w.copy_(ints(wanted))
        graph.replay()
        want = ref.reserve(b.table, held, wanted, b.stack, b.free, 16, T, b.pages)
        b.free = want[4]
        assert [o.tolist() for o in outs] == list(want[:4])
        assert b.gpu[0].tolist() == b.table and b.gpu[1].tolist() == b.stack and b.gpu[2].item() == b.free
        if want[1][-1] > T:  # more tokens than there is room for is reported
            reported += 1
            with pytest.raises(A.AttnError, match="tables"):
                A.attn_check_status()
        A.attn_check_status()
        held, wanted = want[0], [(x * 7 + 5) % 80 for x in want[0]]
    assert 0 < reported < 4


@pytest.mark.parametrize("T", [1023, 1024, 1025, 40959, 40960, 40961])
def test_tokens_at_the_kernels_borders(A, T):
    """Around the numbers of tokens from which a cluster, and then a kernel for the slots, is used; some sequences end."""
    page, n = 32, 6
    held = [5, 0, 700, 33, 64, 4000]
    new = [T // 5, 0, T - T // 5 - T // 7, 0, T // 7, 0]
    wanted = [h + x for h, x in zip(held, new)]
    wanted[3] = wanted[5] = 0
    books = Books(held, page, -(-max(held + wanted) // page) + 2, free=-(-T // page) + n, seed=T)
    start = [list(r) for r in books.table], books.free
    lens = books.step(A, held, wanted, T)[0].tolist()
    assert lens == wanted
    books.step(A, lens, held, new_tokens(lens, held))
    assert (books.table, books.free) == start
    A.attn_check_status()


@pytest.mark.parametrize("n,width", [(4, 4096), (4, 4097), (300, 55), (1, 16384), (1, 16385)])
def test_rooms_at_the_kernels_border(A, n, width):
    """Around the room for pages from which a cluster is used: all of it is taken, then given back."""
    page = 16
    held = [7 * b % 40 for b in range(n)]
    full = [width * page - (b % 16) for b in range(n)]
    books = Books(held, page, width, free=n * width, seed=n)
    T = new_tokens(held, full)
    lens = books.step(A, held, full, T)[0].tolist()
    books.step(A, lens, [0] * n, 0)
    books.step(A, [0] * n, [b % 3 for b in range(n)], n)  # few tokens in a wide table
    A.attn_check_status()


def test_two_at_once(A):
    """Steps of two pools on two streams at the same time."""
    held, wanted = lengths(700, 300, 5)
    T = new_tokens(held, wanted)
    both = [Books(held, 16, 21, free=700 + 50 * i, seed=i) for i in range(2)]
    wants = [ref.reserve(b.table, held, wanted, b.stack, b.free, 16, T, b.pages) for b in both]
    args = ints(held), ints(wanted)
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    gots = []
    for b, s in zip(both, streams):
        with torch.cuda.stream(s):
            gots.append(A.attn_cache_reserve(b.gpu[0], *args, *b.gpu[1:], 16, T))
    torch.cuda.synchronize()
    for b, got, want in zip(both, gots, wants):
        assert [g.tolist() for g in got] == list(want[:4])
        assert b.gpu[0].tolist() == b.table and b.gpu[1].tolist() == b.stack and b.gpu[2].item() == want[4]
    A.attn_check_status()


def test_without_the_tensor_binding(A, monkeypatch):
    """The call through ctypes, and host memory, which both ways refuse."""
    from precision_numerics_gb300 import attn

    held, wanted = [20, 5, 0], [50, 0, 17]
    T = new_tokens(held, wanted)
    for binding in (attn._BINDING, attn._NoBinding):
        monkeypatch.setattr(attn, "_BINDING", binding)
        Books(held, 16, 5, free=9).step(A, held, wanted, T)
        Books(held, 16, 5, free=9).step(A, held, wanted, T, slots=torch.zeros(T, dtype=torch.int32, device="cuda"))
        table, stack, free = Books(held, 16, 5, free=9).gpu
        for args in ((table.cpu(), ints(held), ints(wanted), stack, free), (table, ints(held), ints(wanted), stack.cpu(), free),
                     (table, ints(held).cpu().pin_memory(), ints(wanted), stack, free)):
            with pytest.raises(ValueError):
                A.attn_cache_reserve(*args, 16, T)
        with pytest.raises(ValueError, match="T must"):
            A.attn_cache_reserve(table, ints(held), ints(wanted), stack, free, 16, -1)
    A.attn_check_status()
