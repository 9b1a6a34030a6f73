"""Serving operators on the GPU against their plain 64-bit forms."""
import math

import pytest

import serving_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def A(cuda_device):
    from precision_numerics_gb300 import attn, build
    build.build()
    return attn


def normal(shape, seed, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sums(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------- prompt
def check_prompt(q, k, v, lens, causal, scale, o, lse):
    H, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    o, lse = o.cpu(), lse.cpu()
    at = 0
    for n in lens:
        last = list(range(n)) if causal else [n - 1] * n
        for h in range(H):
            kv = h // (H // Hkv)
            r, rl, a, size = ref.attention(q[at:at + n, h], k[at:at + n, kv], v[at:at + n, kv], scale, last)
            bound = ref.output_bound(r, a, size, d, 2.0 ** -8)
            assert ((o[at:at + n, h].double() - r).abs() <= bound).all(), (at, n, h)
            assert ((lse[at:at + n, h].double() - rl).abs() <= ref.lse_bound(rl, size, d)).all(), (at, n, h)
        at += n


LENS = [
    [1],
    [128],
    [129],
    [5, 0, 127, 1, 0, 64, 255, 257],
    [0, 0, 3],
    [300, 17, 513, 40],
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (8, 2), (6, 2), (10, 2), (14, 2), (64, 1)])
def test_prompt(A, heads, d, causal):
    H, Hkv = heads
    for i, lens in enumerate(LENS):
        T = sum(lens)
        q, k, v = normal((T, H, d), 3 * i), normal((T, Hkv, d), 3 * i + 1), normal((T, Hkv, d), 3 * i + 2)
        plan = A.attn_varlen_plan(ints(sums(lens)), T, H, Hkv, causal=causal)
        o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan, causal=causal)
        A.attn_check_status()
        check_prompt(q, k, v, lens, causal, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_views_and_foreign_rows(A, d):
    """q, k, v as views of one projection's output; a whole sequence of NaN and rows of NaN behind
    the last sequence reach nothing, and rows of no sequence stay as they were."""
    H, Hkv, lens = 6, 3, [70, 33, 200, 131]
    T, cu = 500, sums(lens)
    qkv = normal((T, H + 2 * Hkv, d), 5)
    qkv[cu[1]:cu[2]] = torch.nan
    qkv[cu[4]:] = torch.inf
    x = qkv.cuda()
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    o = torch.full((T, H, d), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    for causal in (True, False):
        plan = A.attn_varlen_plan(ints(cu), T, H, Hkv, causal=causal)
        A.attn_varlen_fwd(q, k, v, plan, scale=0.3, causal=causal, o=o, lse=lse)
        A.attn_check_status()
        assert (o[cu[4]:] == 7).all() and (lse[cu[4]:] == 7).all()
        for b in (0, 2, 3):
            s = slice(cu[b], cu[b + 1])
            check_prompt(qkv[s, :H], qkv[s, H:H + Hkv], qkv[s, H + Hkv:], [lens[b]], causal, 0.3, o[s], lse[s])


def test_prompt_many_short_and_one_long(A):
    """More items than CTAs: several rounds of the list, mixed weights."""
    H, Hkv, d = 8, 4, 128
    lens = [2, 1, 9, 30] * 60 + [2500] + [77] * 20
    T = sum(lens)
    q, k, v = normal((T, H, d), 0), normal((T, Hkv, d), 1), normal((T, Hkv, d), 2)
    plan = A.attn_varlen_plan(ints(sums(lens)), T, H, Hkv)
    o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan)
    A.attn_check_status()
    check_prompt(q, k, v, lens, True, 1 / math.sqrt(d), o, lse)


def test_prompt_matches_the_square_forward(A):
    """Sequences of one length, ungrouped: the same problem as attn_fwd, within both roundings."""
    B, H, N, d = 3, 4, 257, 128
    q, k, v = (normal((B, H, N, d), s).cuda() for s in range(3))
    o0, lse0 = A.attn_fwd(q, k, v, causal=True)
    pack = lambda x: x.transpose(1, 2).reshape(B * N, H, d).contiguous()  # noqa: E731
    plan = A.attn_varlen_plan(ints([0, N, 2 * N, 3 * N]), B * N, H, H)
    o, lse = A.attn_varlen_fwd(pack(q), pack(k), pack(v), plan)
    # The same tiles in the same order: the same bits.
    assert torch.equal(o, pack(o0)) and torch.equal(lse, lse0.transpose(1, 2).reshape(B * N, H))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,d,lens", [((2, 2), 64, [385]), ((8, 2), 128, [498, 385, 384, 1, 513, 0, 70]),
                                          ((5, 1), 64, [640, 129, 900]), ((7, 1), 128, [1500, 3]),
                                          ((3, 3), 128, [511, 512, 640]), ((64, 1), 64, [400, 130])])
def test_prompt_split_items(A, heads, d, lens, causal):
    """Few items: the two tiles of a CTA share an item's keys where it has enough; CTAs with several
    items, split ones and others; rows behind the sequences are left as they are; the same bits twice."""
    H, Hkv = heads
    T = sum(lens)
    q, k, v = normal((T + 9, H, d), 1), normal((T + 9, Hkv, d), 2), normal((T + 9, Hkv, d), 3)
    v[T:] = torch.nan
    plan = A.attn_varlen_plan(ints(sums(lens)), T + 9, H, Hkv, causal=causal)
    got = []
    for _ in range(2):
        o = torch.full((T + 9, H, d), 7.0, dtype=BF, device="cuda")
        lse = torch.full((T + 9, H), 7.0, device="cuda")
        got.append(A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan, causal=causal, o=o, lse=lse))
        A.attn_check_status()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (got[0][0][T:] == 7).all() and (got[0][1][T:] == 7).all()
    check_prompt(q, k, v, lens, causal, 1 / math.sqrt(d), *got[0])


def test_prompt_large_scores(A):
    """Scores of several hundred: one key takes all the weight in most rows."""
    lens, H, Hkv, d = [150, 260], 4, 2, 64
    T = sum(lens)
    q, k, v = normal((T, H, d), 0) * 8, normal((T, Hkv, d), 1) * 8, normal((T, Hkv, d), 2)
    plan = A.attn_varlen_plan(ints(sums(lens)), T, H, Hkv)
    o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan)
    check_prompt(q, k, v, lens, True, 1 / math.sqrt(d), o, lse)


def test_prompt_refusals(A):
    H, Hkv, d = 4, 2, 64
    q, k, v = normal((30, H, d), 0).cuda(), normal((30, Hkv, d), 1).cuda(), normal((30, Hkv, d), 2).cuda()
    plan = A.attn_varlen_plan(ints([0, 30]), 30, H, Hkv)
    with pytest.raises(ValueError):
        A.attn_varlen_fwd(q.float(), k, v, plan)
    with pytest.raises(ValueError):
        A.attn_varlen_fwd(q, k, v[:29], plan)
    with pytest.raises(ValueError):
        A.attn_varlen_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, plan)
    with pytest.raises(ValueError):
        A.attn_varlen_fwd(q[:, :3], k, v, plan)
    # A plan of another batch or mask computes nothing and says so.
    o = torch.full((30, H, d), 7.0, dtype=BF, device="cuda")
    for other in (A.attn_varlen_plan(ints([0, 30]), 30, H, Hkv, causal=False),
                  A.attn_varlen_plan(ints([0, 29]), 29, H, Hkv), torch.zeros_like(plan)):
        A.attn_varlen_fwd(q, k, v, other, o=o)
        with pytest.raises(A.AttnError, match="INVALID_ARG"):
            A.attn_check_status()
        assert (o == 7).all()
    # Lengths that run backwards or past T are cut to the tensors.
    for cu in ([0, 40], [0, 20, 10, 30], [-5, 30], [0, 30, 0, 30, 0, 30, 0, 30]):
        p = A.attn_varlen_plan(ints(cu), 30, H, Hkv)
        A.attn_varlen_fwd(q, k, v, p)
        with pytest.raises(A.AttnError, match="INVALID_ARG"):
            A.attn_check_status()
    A.attn_check_status()


# -------------------------------------------------------------------- cache
class Cache:
    def __init__(self, pages, Hkv, page, d, tables, seed=0, width=None):
        g = torch.Generator().manual_seed(seed)
        self.codes = [torch.randint(-127, 128, (pages, Hkv, page, d), generator=g, dtype=torch.int8) for _ in range(2)]
        self.scales = [torch.rand((pages, Hkv), generator=g) * 0.02 + 0.001 for _ in range(2)]
        self.tables = tables
        width = width or max(1, max(len(t) for t in tables))
        self.table = ints([list(t) + [-1] * (width - len(t)) for t in tables])
        self.upload()

    def upload(self):
        self.gpu = (self.codes[0].cuda(), self.codes[1].cuda(), self.scales[0].cuda(), self.scales[1].cuda(), self.table)

    def equal(self):
        """The GPU's cache is this one, bit for bit, pages of nobody included."""
        return all(torch.equal(a, b.cpu()) for a, b in zip(self.codes + self.scales, self.gpu))

    def append(self, rows, cu, starts):
        for i in range(2):
            for b, t in enumerate(self.tables):
                ref.append(rows[i][cu[b]:cu[b + 1]], self.codes[i], self.scales[i], t, starts[b])

    def values(self, i, b, n):
        return ref.cached(self.codes[i], self.scales[i], self.tables[b], n)


def scattered(counts, seed, spare=3):
    """Disjoint tables of so many pages each, in scattered order; the pool's size."""
    total = sum(counts) + spare
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    out, at = [], 0
    for n in counts:
        out.append(order[at:at + n])
        at += n
    return out, total


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append(A, page, d):
    """Fresh pages, pages begun earlier whose scale grows or stays, several pages at once, nothing;
    a second call with the same rows changes nothing more."""
    Hkv = 3
    starts = [0, 5, page - 1, page, 3 * page + 2, 7, 2, 0]
    lens = [1, 1, 2, page, 2 * page + 3, 0, page + 1, 3 * page]
    tables, pages = scattered([-(-(s + n) // page) for s, n in zip(starts, lens)], 1)
    c = Cache(pages, Hkv, page, d, tables)
    T, cu = sum(lens), sums(lens)
    rows = [normal((T, Hkv, d), 1), normal((T, Hkv, d), 2) * 0.01]  # V's new rows are small: its scales stay
    c.append(rows, cu, starts)
    args = (rows[0].cuda(), rows[1].cuda(), *c.gpu, ints(cu), ints(starts))
    for _ in range(2):
        A.attn_cache_append_int8(*args)
        A.attn_check_status()
        assert c.equal()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_append_few_rows(A, page, d):
    """A step: a row or a few a sequence, more heads than warps, scales that grow by little and by much
    (held codes on and next to the border), special values."""
    Hkv = 11
    starts = [0, 1, 5, page - 1, 2 * page, 3 * page - 2, 9, 0, 13, 15]
    lens = [1, 1, 2, 2, 1, 5, 0, page + 2, 1, 1]
    tables, pages = scattered([-(-(s + n) // page) for s, n in zip(starts, lens)], 21)
    c = Cache(pages, Hkv, page, d, tables)
    T, cu = sum(lens), sums(lens)
    assert T <= 8 * len(lens) or page > 16
    g = torch.Generator().manual_seed(9)
    rows = [normal((T, Hkv, d), i) * torch.exp(2 * torch.randn(T, Hkv, 1, generator=g)).to(BF) for i in (1, 2)]
    rows[0][2, 3, 4], rows[0][2, 4, 4], rows[1][2, 5, 0] = torch.nan, torch.inf, -torch.inf
    c.scales[0][tables[2][0]] = 2.0 ** -6  # doubled exactly: every odd code is a tie
    rows[0][2:4] = 0
    rows[0][2:4, :, 7] = 127 * 2.0 ** -5
    c.upload()
    c.append(rows, cu, starts)
    args = (rows[0].cuda(), rows[1].cuda(), *c.gpu, ints(cu), ints(starts))
    for _ in range(2):
        A.attn_cache_append_int8(*args)
        A.attn_check_status()
        assert c.equal()


def test_append_views_zeros_and_special_values(A):
    """Rows of a fused projection; rows of zeros on a fresh page; a NaN and infinities stay out of the
    scale and become 0 and +-127; tiny and huge values."""
    page, d, Hkv, lens, starts = 16, 64, 2, [3, 20, 18], [0, 9, 16]
    tables, pages = scattered([1, 2, 3], 2)
    c = Cache(pages, Hkv, page, d, tables)
    T, cu = sum(lens), sums(lens)
    qkv = normal((T, 3 * Hkv, d), 3)
    qkv[:3] = 0
    qkv[4, Hkv, 5] = torch.nan
    qkv[5, Hkv, 6], qkv[6, Hkv, 7] = torch.inf, -torch.inf
    qkv[cu[2]:, Hkv] *= 1e30
    qkv[cu[2]:, 2 * Hkv] *= 1e-30
    rows = [qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]]
    c.append(rows, cu, starts)
    x = qkv.cuda()
    A.attn_cache_append_int8(x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], *c.gpu, ints(cu), ints(starts))
    A.attn_check_status()
    assert c.equal()


def test_append_values_on_the_border(A):
    """x = (2 k + 1) / 2 steps of the scale: ties of the exact quotient, or next to them, where the
    scale a / 127 is not a power of two."""
    page, d = 32, 128
    tables, pages = scattered([4], 3)
    c = Cache(pages, 1, page, d, tables)
    rows = torch.zeros((4 * page, 1, d), dtype=BF)
    for j, a in enumerate((254.0, 1.9921875, 3.0, 200.0)):
        block = rows[j * page:(j + 1) * page].view(-1)
        block[:] = (torch.arange(page * d) % 509 - 254.0).to(BF) * (a / 254.0)
        block[0] = a
        block[1:40] = torch.tensor(a / 2)
    c.append([rows, rows], [0, 4 * page], [0])
    A.attn_cache_append_int8(rows.cuda(), rows.cuda(), *c.gpu, ints([0, 4 * page]), ints([0]))
    assert c.equal()


@pytest.mark.parametrize("rows", [1, 20])
def test_append_rescales_the_lowest_code(A, rows):
    """Held codes of -128, which the cache's own writes never leave, are clamped like all others
    when their page's scale grows a little."""
    page, d, start = 32, 64, 7
    tables, pages = scattered([1], 5)
    c = Cache(pages, 1, page, d, tables)
    for codes in c.codes:
        codes[:, :, :start, ::3] = -128
    c.scales = [torch.full((pages, 1), 2.0125 / 127) for _ in range(2)]
    c.upload()
    new = torch.full((rows, 1, d), 2.015625, dtype=BF)
    c.append([new, new], [0, rows], [start])
    A.attn_cache_append_int8(new.cuda(), new.cuda(), *c.gpu, ints([0, rows]), ints([start]))
    A.attn_check_status()
    assert c.equal() and all((x[tables[0][0], 0, :start].amin() == -127) for x in c.codes)


def test_append_many_sequences(A):
    """More sequences than a CTA scans at a time, one token each, as a decoding step does."""
    B, Hkv, page, d = 300, 2, 16, 64
    starts = [(7 * b) % 40 for b in range(B)]
    tables, pages = scattered([s // page + 1 for s in starts], 4)
    c = Cache(pages, Hkv, page, d, tables)
    rows = [normal((B, Hkv, d), 1), normal((B, Hkv, d), 2)]
    c.append(rows, list(range(B + 1)), starts)
    A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *c.gpu, ints(list(range(B + 1))), ints(starts))
    A.attn_check_status()
    assert c.equal()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_read(A, page, d, dtype):
    Hkv, starts, lens = 3, [0, 5, 40, page - 1], [1, 0, 3 * page + 1, 2]
    tables, pages = scattered([-(-(s + n) // page) for s, n in zip(starts, lens)], 5)
    c = Cache(pages, Hkv, page, d, tables)
    k, v = A.attn_cache_read_int8(*c.gpu, ints(sums(lens)), ints(starts), sum(lens), dtype=dtype)
    A.attn_check_status()
    for i, got in enumerate((k, v)):
        want = torch.cat([c.values(i, b, s + n)[s:] for b, (s, n) in enumerate(zip(starts, lens))])
        # A product of an 8-bit and a 24-bit number rounded to FP32, then to the type.
        assert torch.equal(got.cpu(), want.float().to(dtype))


def test_bad_pages_are_reported_and_skipped(A):
    page, d, Hkv = 16, 64, 2
    c = Cache(6, Hkv, page, d, [[0, 1], [2, 3]])
    table = ints([[0, 99], [-7, 3]])
    gpu = (*c.gpu[:4], table)
    rows = [normal((64, Hkv, d), 1), normal((64, Hkv, d), 2)]
    for i in range(2):  # the pages within range are written
        ref.append(rows[i][:16], c.codes[i], c.scales[i], [0], 0)
        ref.append(rows[i][48:], c.codes[i], c.scales[i], [9, 3], 16)
    A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *gpu, ints([0, 32, 64]), ints([0, 0]))
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    assert c.equal()
    k, _ = A.attn_cache_read_int8(*gpu, ints([0, 32, 64]), ints([0, 0]), 64, dtype=torch.float32)
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    assert (k[16:48] == 0).all() and torch.equal(k[:16].cpu(), c.values(0, 0, 16).float())
    # Lengths that run backwards or past T, negative starts.
    for cu, starts in (([0, 40, 30], [0, 0]), ([0, 10, 70], [0, 0]), ([0, 16, 16], [-1, 0])):
        A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *c.gpu, ints(cu), ints(starts))
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
        A.attn_cache_read_int8(*c.gpu, ints(cu), ints(starts), 64)
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
    # Beyond the table's width.
    A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *c.gpu, ints([0, 32, 64]), ints([30, 2**31 - 1]))
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    A.attn_check_status()


# ------------------------------------------------------------------- decode
def check_decode(c, q, lens, scale, o, lse, shown=None):
    B, n_q, H, d = q.shape
    Hkv = c.codes[0].shape[1]
    G = H // Hkv
    o, lse = o.cpu(), lse.cpu()
    for b, n in enumerate(lens):
        if shown is not None and b not in shown:
            continue
        k, v = c.values(0, b, n), c.values(1, b, n)
        last = [n - n_q + i for i in range(n_q) for _ in range(G)]
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            r, rl, a, size = ref.attention(q[b, :, hs].reshape(-1, d), k[:, h], v[:, h], scale, last)
            got, gl = o[b, :, hs].reshape(-1, d).double(), lse[b, :, hs].reshape(-1).double()
            # P vs is held in FP16 as p 2^15 vs / R, p <= 1 relative to a running maximum no larger than
            # the row's, R < 2 max vs: relative 2^-11, and below 2^-14 absolute 2^-25.  The latter is
            # 2^-40 R |c| <= 2^-39 * 127 * max vs a key, over a row sum of at least 1: what a row
            # shows whose large probabilities all meet a code of 0.
            ids = c.tables[b][:-(-n // c.codes[1].shape[2])]
            least = n * 127 * 2.0 ** -39 * float(c.scales[1][ids, h].max()) if n else 0.0
            bound = ref.output_bound(r, a, size, d, 2.0 ** -11) + least
            assert ((got - r).abs() <= bound).all(), (b, h)
            dead = rl.isinf()
            assert (got[dead] == 0).all() and (gl[dead] == -torch.inf).all()
            assert ((gl - rl)[~dead].abs() <= ref.lse_bound(rl, size, d)[~dead]).all(), (b, h)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,n_q", [((1, 1), 1), ((4, 4), 1), ((8, 2), 1), ((14, 2), 1), ((12, 3), 3), ((32, 2), 1),
                                       ((10, 2), 7), ((64, 1), 2)])
def test_decode(A, heads, n_q, page, d):
    H, Hkv = heads
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 300, 1000]
    tables, pages = scattered([-(-n // page) for n in lens], 7)
    c = Cache(pages, Hkv, page, d, tables)
    q = normal((len(lens), n_q, H, d), 1)
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    check_decode(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("lens", [[9000], [1, 20000, 3], [4000] * 3 + [0, 40]])
def test_decode_long(A, lens):
    """Few long sequences: the keys are split over CTAs and joined."""
    H, Hkv, d, page = 8, 2, 128, 64
    tables, pages = scattered([-(-n // page) for n in lens], 8)
    c = Cache(pages, Hkv, page, d, tables)
    for n_q in (1, 5):
        q = normal((len(lens), n_q, H, d), 1) * 2
        o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens), scale=0.05)
        A.attn_check_status()
        check_decode(c, q, lens, 0.05, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_short(A, page, d):
    """A table too narrow for the keys to be split: one CTA a sequence and key head."""
    H, Hkv, lens = 6, 3, [0, 1, 16, 17, 31, 250, 512, 499]
    tables, pages = scattered([-(-n // page) for n in lens], 13)
    c = Cache(pages, Hkv, page, d, tables)
    for n_q in (1, 9):
        q = normal((len(lens), n_q, H, d), 1)
        o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
        A.attn_check_status()
        check_decode(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d,G,n_q", [(64, 1, 1), (64, 4, 4), (128, 2, 1), (128, 5, 4), (128, 8, 4), (64, 20, 2)])
@pytest.mark.parametrize("B", [1, 19, 23, 31, 47, 70])
def test_decode_shared_by_clusters(A, B, d, G, n_q):
    """Segments shared by 2 to 8 CTAs each, as their number allows; sequences of fewer tiles than
    CTAs, and empty ones; the same bits twice."""
    Hkv, page, most = 2, 32, 700
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, most + 1, (B,), generator=g).tolist()
    lens[0] = most
    lens[1:6] = [0, 1, 33, 64, 250][:B - 1]
    tables, pages = scattered([-(-n // page) for n in lens], 18)
    c = Cache(pages, Hkv, page, d, tables)
    q = normal((B, n_q, Hkv * G, d), 1)
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    again, lse_again = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    assert torch.equal(o, again) and torch.equal(lse, lse_again)
    check_decode(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("most,page", [(2000, 16), (9000, 128)])
def test_decode_ragged_batch(A, most, page):
    """More sequences than a CTA scans at a time, among them empty ones; runs of tiles that begin and
    end anywhere in a segment, hold several, or lie inside one."""
    H, Hkv, d, B = 4, 2, 64, 171
    g = torch.Generator().manual_seed(most)
    lens = torch.randint(0, 70, (B,), generator=g).tolist()
    lens[::9] = torch.randint(0, most, (len(lens[::9]),), generator=g).tolist()
    lens[5:8] = lens[-3:] = [0, 0, 0]
    tables, pages = scattered([-(-n // page) for n in lens], 14)
    c = Cache(pages, Hkv, page, d, tables, width=-(-most // page))
    q = normal((B, 1, H, d), 1)
    o = torch.full((B, 1, H, d), 7.0, dtype=BF, device="cuda")
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens), o=o)
    A.attn_check_status()
    check_decode(c, q, lens, 1 / math.sqrt(d), o, lse)


def test_decode_scales_of_every_size(A):
    """Pages whose value scales differ by 2^60, pages of zeros, keys of zero scale, queries of zeros
    and of extreme size."""
    H, Hkv, d, page, lens = 4, 1, 64, 16, [200, 333]
    tables, pages = scattered([-(-n // page) for n in lens], 9)
    c = Cache(pages, Hkv, page, d, tables)
    c.scales[1][:] *= 2.0 ** torch.randint(-30, 31, c.scales[1].shape, generator=torch.Generator().manual_seed(3))
    c.scales[1][tables[0][2]] = 0
    c.scales[0][tables[0][3]] = 0
    c.upload()
    q = normal((2, 1, H, d), 1)
    q[0, 0, 1] = 0
    q[0, 0, 2] *= 1e-30
    q[0, 0, 3, 1:] *= 1e-6
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    check_decode(c, q, lens, 1 / math.sqrt(d), o, lse)


@pytest.mark.parametrize("d,n_q", [(64, 1), (128, 1), (128, 5)])
@pytest.mark.parametrize("lens", [[40, 300], [3000, 9, 20000]])
def test_decode_largest_values_and_nan_rows(A, lens, d, n_q):
    """Value scales up to 2^118, whose sums over the keys leave the type; a NaN in a query stays in its
    row of O and LSE."""
    H, Hkv, page = 4, 2, 32
    tables, pages = scattered([-(-n // page) for n in lens], 17)
    c = Cache(pages, Hkv, page, d, tables)
    c.scales[1][:] = 2.0 ** torch.randint(90, 119, c.scales[1].shape, generator=torch.Generator().manual_seed(4))
    c.upload()
    q = normal((len(lens), n_q, H, d), 1)
    bad = q.clone()
    bad[1, n_q - 1, 2, 3] = torch.nan
    o, lse = A.attn_decode_int8(bad.cuda(), *c.gpu, ints(lens))
    assert o[1, n_q - 1, 2].isnan().all() and lse[1, n_q - 1, 2].isnan()
    good, good_lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints(lens))
    A.attn_check_status()
    check_decode(c, q, lens, 1 / math.sqrt(d), good, good_lse)
    o[1, n_q - 1, 2], lse[1, n_q - 1, 2] = good[1, n_q - 1, 2], good_lse[1, n_q - 1, 2]
    assert torch.equal(o, good) and torch.equal(lse, good_lse)


def test_decode_shared_pages_views_and_bad_lengths(A):
    """Two sequences share their first pages; q is a view of a fused projection's output; rows of the
    last page behind the length do not count; a length past the table and a bad page are reported."""
    H, Hkv, d, page = 8, 2, 128, 32
    c = Cache(12, Hkv, page, d, [[4, 7, 1], [4, 7, 9, 2], [5]])
    lens = [70, 100, 20]
    qkv = normal((3, 1, H + 2 * Hkv, d), 2)
    q = qkv[:, :, :H]
    o, lse = A.attn_decode_int8(qkv.cuda()[:, :, :H], *c.gpu, ints(lens))
    A.attn_check_status()
    check_decode(c, q, lens, 1 / math.sqrt(d), o, lse)
    o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints([70, 100, 50]))  # sequence 2 has one page
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    check_decode(c, q, [70, 100, 32], 1 / math.sqrt(d), o, lse)  # the missing page's positions are not seen
    for wrong in (10**6, -3):
        o, lse = A.attn_decode_int8(q.cuda(), *c.gpu, ints([70, 100, wrong]))
        with pytest.raises(A.AttnError, match="out of range"):
            A.attn_check_status()
        check_decode(c, q, lens, 1 / math.sqrt(d), o, lse, shown=(0, 1))
    A.attn_check_status()


def test_decode_refusals(A):
    c = Cache(4, 2, 16, 64, [[0, 1]])
    q = normal((1, 1, 4, 64), 0).cuda()
    with pytest.raises(ValueError):
        A.attn_decode_int8(q.half(), *c.gpu, ints([5]))
    with pytest.raises(ValueError):
        A.attn_decode_int8(q, *c.gpu, ints([5, 6]))
    with pytest.raises(ValueError):
        A.attn_decode_int8(q, c.gpu[0].float(), *c.gpu[1:], ints([5]))
    with pytest.raises(ValueError):
        A.attn_decode_int8(q, *c.gpu[:4], c.gpu[4].long(), ints([5]))
    with pytest.raises(A.AttnError, match="UNSUPPORTED"):
        A.attn_decode_int8(normal((1, 1, 4, 64), 0).cuda(), c.gpu[0][:, :, :8].contiguous(),
                           c.gpu[1][:, :, :8].contiguous(), *c.gpu[2:], ints([5]))
    with pytest.raises(A.AttnError, match="multiple of H_kv"):
        A.attn_decode_int8(normal((1, 1, 5, 64), 0).cuda(), *c.gpu, ints([5]))


def test_cache_beyond_four_gib(A):
    """Pages whose bytes lie past 2^32 (and whose rows' number times d does)."""
    Hkv, page, d, H = 8, 128, 128, 16
    pages = 2 ** 32 // (Hkv * page * d) + 40
    last = [pages - 1, pages - 3, pages - 2, 5, pages - 7]
    k_cache, v_cache = (torch.zeros((pages, Hkv, page, d), dtype=torch.int8, device="cuda") for _ in range(2))
    k_scale, v_scale = (torch.zeros((pages, Hkv), device="cuda") for _ in range(2))
    c = Cache(5, Hkv, page, d, [[0, 1, 2, 3, 4]])  # the same five pages, small enough for the host
    for i, (codes, scale) in enumerate(((k_cache, k_scale), (v_cache, v_scale))):
        codes[last], scale[last] = c.codes[i].cuda(), c.scales[i].cuda()
    gpu = k_cache, v_cache, k_scale, v_scale, ints([last])
    n, new = 500, 20
    rows = [normal((new, Hkv, d), 1), normal((new, Hkv, d), 2)]
    c.append(rows, [0, new], [n])
    A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *gpu, ints([0, new]), ints([n]))
    A.attn_check_status()
    assert all(torch.equal(x[last].cpu(), y) for x, y in zip(gpu, c.codes + c.scales))
    k, _ = A.attn_cache_read_int8(*gpu, ints([0, n + new]), ints([0]), n + new, dtype=torch.float32)
    assert torch.equal(k.cpu(), c.values(0, 0, n + new).float())
    q = normal((1, 1, H, d), 3)
    o, lse = A.attn_decode_int8(q.cuda(), *gpu, ints([n + new]))
    A.attn_check_status()
    check_decode(c, q, [n + new], 1 / math.sqrt(d), o, lse)


# ----------------------------------------------------------------- together
def test_prompt_then_steps(A):
    """A serving run: prompts attend and enter the cache, then tokens are appended and attend over it,
    two at a time, through one captured graph replayed on new inputs on a stream of its own."""
    H, Hkv, d, page, steps = 8, 2, 128, 32, 6
    lens = [45, 64, 1, 200]
    B, T, cu = len(lens), sum(lens), sums(lens)
    tables, pages = scattered([-(-(n + 2 * steps) // page) for n in lens], 11)
    c = Cache(pages, Hkv, page, d, tables)
    q, k, v = normal((T, H, d), 1), normal((T, Hkv, d), 2), normal((T, Hkv, d), 3)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        plan = A.attn_varlen_plan(ints(cu), T, H, Hkv)
        o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan)
        A.attn_cache_append_int8(k.cuda(), v.cuda(), *c.gpu, ints(cu), ints([0] * B))
        A.attn_check_status()
        check_prompt(q, k, v, lens, True, 1 / math.sqrt(d), o, lse)
        c.append([k, v], cu, [0] * B)
        assert c.equal()

        new = torch.zeros((B, 2, H + 2 * Hkv, d), dtype=BF, device="cuda")  # a fused projection's output
        held, total = ints([0] * B), ints([0] * B)
        step_cu = ints([2 * b for b in range(B + 1)])
        o = torch.zeros((B, 2, H, d), dtype=BF, device="cuda")
        lse = torch.zeros((B, 2, H), device="cuda")
        ws = torch.empty(max(1, A.attn_decode_int8_workspace_bytes(B, 2, H, Hkv, d, page, c.table.shape[1])),
                         dtype=torch.uint8, device="cuda")

        def step():
            rows = new.view(2 * B, H + 2 * Hkv, d)
            A.attn_cache_append_int8(rows[:, H:H + Hkv], rows[:, H + Hkv:], *c.gpu, step_cu, held)
            A.attn_decode_int8(new[:, :, :H], *c.gpu, total, o=o, lse=lse, workspace=ws)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for s in range(steps):
            x = normal((B, 2, H + 2 * Hkv, d), 20 + s) * (1 + s)
            new.copy_(x)
            held.copy_(ints([n + 2 * s for n in lens]))
            total.copy_(ints([n + 2 * s + 2 for n in lens]))
            graph.replay()
            A.attn_check_status()
            rows = x.view(2 * B, H + 2 * Hkv, d)
            c.append([rows[:, H:H + Hkv], rows[:, H + Hkv:]], [2 * b for b in range(B + 1)], [n + 2 * s for n in lens])
            assert c.equal()
            check_decode(c, x[:, :, :H], [n + 2 * s + 2 for n in lens], 1 / math.sqrt(d), o, lse)


def test_prompts_in_a_graph(A):
    """The plan and the attention captured once, replayed on other lengths of the same total."""
    H, Hkv, d, T = 4, 1, 64, 400
    x = normal((T, H + 2 * Hkv, d), 1)
    cu = ints([0, 100, 200, 300, 400])
    o, lse = torch.zeros((T, H, d), dtype=BF, device="cuda"), torch.zeros((T, H), device="cuda")
    plan = torch.empty(A.attn_varlen_plan_bytes(4, T, H, Hkv), dtype=torch.uint8, device="cuda")
    y = x.cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        A.attn_varlen_plan(cu, T, H, Hkv, plan=plan)
        A.attn_varlen_fwd(y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:], plan, o=o, lse=lse)
    for lens in ([100] * 4, [399, 0, 0, 1], [1, 129, 128, 142]):
        cu.copy_(ints(sums(lens)))
        graph.replay()
        A.attn_check_status()
        check_prompt(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], lens, True, 1 / math.sqrt(d), o, lse)


def test_the_same_call_twice_gives_the_same_bits(A):
    H, Hkv, d, page, lens = 8, 2, 128, 64, [5000, 3, 700]
    tables, pages = scattered([-(-n // page) for n in lens], 12)
    c = Cache(pages, Hkv, page, d, tables)
    q = normal((3, 1, H, d), 1).cuda()
    x = normal((900, H + 2 * Hkv, d), 2).cuda()
    plan = A.attn_varlen_plan(ints([0, 500, 900]), 900, H, Hkv)
    first = None
    for _ in range(5):
        got = (*A.attn_decode_int8(q, *c.gpu, ints(lens)),
               *A.attn_varlen_fwd(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], plan))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_calls_with_a_stream_given(A):
    """The binding's two ways, with and without an explicit stream, and a scale that is no float."""
    H, Hkv, d, page, lens = 4, 2, 64, 16, [70, 9]
    T, cu = sum(lens), sums(lens)
    x = normal((T, H + 2 * Hkv, d), 1).cuda()
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    tables, pages = scattered([5, 1], 3)
    results = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, scale in ((None, 1.0), (side, 1.0), (side.cuda_stream, 1.0), (None, 1)):
        c = Cache(pages, Hkv, page, d, tables)
        torch.cuda.synchronize()
        plan = A.attn_varlen_plan(ints(cu), T, H, Hkv, stream=stream)
        torch.cuda.synchronize()
        got = [*A.attn_varlen_fwd(q, k, v, plan, scale=scale, stream=stream)]
        args = ints(cu), ints([0, 0]), ints(lens)
        qd = q[[lens[0] - 1, T - 1]].view(2, 1, H, d)
        torch.cuda.synchronize()
        assert A.attn_cache_append_int8(k, v, *c.gpu, *args[:2], stream=stream)[0] is c.gpu[0]
        got += A.attn_cache_read_int8(*c.gpu, *args[:2], T, stream=stream)
        got += A.attn_decode_int8(qd, *c.gpu, args[2], scale=scale, stream=stream)
        torch.cuda.synchronize()
        results.append(got)
    for got in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], got))
    A.attn_check_status()


def test_memory_of_calls_on_another_stream(A, monkeypatch):
    """What a call on a given stream allocates is memory of that stream: once the call has returned,
    and its tensors are gone, the current stream does not get it while the kernels may still run."""
    H, Hkv, d, page, T = 2, 1, 64, 16, 600
    q, kv = normal((T, H, d), 1).cuda(), normal((T, Hkv, d), 2).cuda()
    tables, pages = scattered([40], 3)
    c = Cache(pages, Hkv, page, d, tables)
    cu, starts, lens = ints([0, T]), ints([0]), ints([T])
    plan = A.attn_varlen_plan(cu, T, H, Hkv)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    used = []
    call = A._call
    monkeypatch.setattr(A, "_call", lambda name, *args: used.extend(
        x for x in args if isinstance(x, int) and x > 1 << 32) or call(name, *args))
    workspace = A.attn_decode_int8_workspace_bytes(1, 1, H, Hkv, d, page, 40)
    calls = (
        (lambda s: A.attn_varlen_plan(cu, T, H, Hkv, stream=s), [A.attn_varlen_plan_bytes(1, T, H, Hkv)]),
        (lambda s: A.attn_varlen_fwd(q, kv, kv, plan, stream=s), [T * H * d * 2, T * H * 4]),
        (lambda s: A.attn_cache_read_int8(*c.gpu, cu, starts, T, stream=s), [T * Hkv * d * 2] * 2),
        (lambda s: A.attn_decode_int8(q[:1, None], *c.gpu, lens, stream=s), [H * d * 2, H * 4, workspace]),
    )
    for run, sizes in calls:
        for stream in (side, side.cuda_stream):
            used.clear()
            run(stream)
            after = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
            assert used and not set(used) & {x.data_ptr() for x in after}
            torch.cuda.synchronize()
    A.attn_check_status()


def test_host_memory_is_refused(A):
    """Pinned host memory among device pointers, in every place but the outputs'."""
    page, d, Hkv = 16, 64, 2
    tables, pages = scattered([1], 3)
    c = Cache(pages, Hkv, page, d, tables)
    rows, q = normal((3, Hkv, d), 1).cuda(), normal((1, 1, 4, d), 2).cuda()
    host = torch.zeros(pages * Hkv * page * d, dtype=torch.int8).pin_memory().data_ptr()
    cu, starts, lens = ints([0, 3]), ints([0]), ints([3])
    o, lse = torch.empty_like(q), torch.empty((1, 1, 4), device="cuda")
    pointers = [x.data_ptr() for x in (rows, rows)], [x.data_ptr() for x in (*c.gpu, cu, starts)]
    for i in range(9):
        p = [*pointers[0], *pointers[1]]
        p[i] = host
        with pytest.raises(A.AttnError, match="is not device memory"):
            A._call("attn_cache_append_int8", *p[:2], Hkv * d, d, Hkv * d, d, *p[2:], 1, 3, Hkv, d, pages, page, 1, 0)
    for i in range(7):
        p = [q.data_ptr(), *(x.data_ptr() for x in (*c.gpu, lens))]
        p[i] = host
        with pytest.raises(A.AttnError, match="is not device memory"):
            A._call("attn_decode_int8", p[0], 4 * d, 4 * d, d, *p[1:], o.data_ptr(), lse.data_ptr(), 1, 1, 4, Hkv, d, pages,
                    page, 1, 0.125, 0, 0, 0)
    A.attn_check_status()


# ------------------------------------------------ sizes, layouts, several calls
def test_thousands_of_sequences(A):
    """More sequences than any kernel holds at a time, many of them empty."""
    H, Hkv, d, page, B = 2, 1, 64, 16, 3000
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 9, (B,), generator=g).tolist()
    lens[2500] = 700
    T, cu = sum(lens), sums(lens)
    q, k, v = normal((T, H, d), 1), normal((T, Hkv, d), 2), normal((T, Hkv, d), 3)
    plan = A.attn_varlen_plan(ints(cu), T, H, Hkv)
    o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan)
    A.attn_check_status()
    some = [b for b in range(0, B, 97)] + [2500, B - 1]
    for b in some:
        s = slice(cu[b], cu[b + 1])
        check_prompt(q[s], k[s], v[s], [lens[b]], True, 1 / math.sqrt(d), o[s], lse[s])
    starts = torch.randint(0, 20, (B,), generator=g).tolist()
    tables, pages = scattered([-(-(s + n) // page) for s, n in zip(starts, lens)], 2)
    c = Cache(pages, Hkv, page, d, tables)
    c.append([k, v], cu, starts)
    A.attn_cache_append_int8(k.cuda(), v.cuda(), *c.gpu, ints(cu), ints(starts))
    A.attn_check_status()
    assert c.equal()
    got, _ = A.attn_cache_read_int8(*c.gpu, ints(cu), ints(starts), T, dtype=torch.float32)
    A.attn_check_status()
    want = torch.cat([c.values(0, b, s + n)[s:] for b, (s, n) in enumerate(zip(starts, lens))])
    assert torch.equal(got.cpu(), want.float())
    held = [s + n for s, n in zip(starts, lens)]
    qd = normal((B, 1, H, d), 4)
    o, lse = A.attn_decode_int8(qd.cuda(), *c.gpu, ints(held))
    A.attn_check_status()
    check_decode(c, qd, held, 1 / math.sqrt(d), o, lse, shown=some)


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_of_seventy_thousand_tokens(A, causal):
    H, Hkv, d, T = 2, 1, 64, 70001
    q, k, v = normal((T, H, d), 1), normal((T, Hkv, d), 2), normal((T, Hkv, d), 3)
    plan = A.attn_varlen_plan(ints([0, T]), T, H, Hkv, causal=causal)
    o, lse = A.attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), plan, causal=causal)
    A.attn_check_status()
    rows = [0, 1, 127, 128, 40000, 65535, 65536, T - 1]
    for h in range(H):
        r, rl, a, size = ref.attention(q[rows, h], k[:, 0], v[:, 0], 1 / math.sqrt(d), rows if causal else [T - 1] * len(rows))
        assert ((o[rows, h].cpu().double() - r).abs() <= ref.output_bound(r, a, size, d, 2.0 ** -8)).all()
        assert ((lse[rows, h].cpu().double() - rl).abs() <= ref.lse_bound(rl, size, d)).all()


def test_head_major_tensors(A):
    """q, k, v stored head by head (token stride below the head stride)."""
    H, Hkv, d, lens = 6, 2, 128, [130, 77]
    T = sum(lens)
    q, k, v = (normal((n, T, d), i).transpose(0, 1) for i, n in enumerate((H, Hkv, Hkv)))
    plan = A.attn_varlen_plan(ints(sums(lens)), T, H, Hkv)
    gq, gk, gv = (x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in (q, k, v))
    assert gq.stride(0) == d
    o, lse = A.attn_varlen_fwd(gq, gk, gv, plan)
    A.attn_check_status()
    check_prompt(q, k, v, lens, True, 1 / math.sqrt(d), o, lse)
    tables, pages = scattered([9, 5], 3)
    c = Cache(pages, Hkv, 16, d, tables)
    c.append([k, v], sums(lens), [0, 0])
    A.attn_cache_append_int8(gk, gv, *c.gpu, ints(sums(lens)), ints([0, 0]))
    assert c.equal()
    qd = q[:2].reshape(2, 1, H, d)
    strided = qd.transpose(0, 2).contiguous().cuda().transpose(0, 2)
    o, lse = A.attn_decode_int8(strided, *c.gpu, ints(lens))
    A.attn_check_status()
    check_decode(c, qd, lens, 1 / math.sqrt(d), o, lse)


def test_batch_without_tokens(A):
    """Sequences that are all empty, with rows of nobody behind them; no rows at all."""
    H, Hkv, d = 4, 2, 64
    q, k = normal((40, H, d), 1).cuda(), normal((40, Hkv, d), 2).cuda()
    o, lse = torch.full((40, H, d), 7.0, dtype=BF, device="cuda"), torch.full((40, H), 7.0, device="cuda")
    plan = A.attn_varlen_plan(ints([0, 0, 0, 0]), 40, H, Hkv)
    A.attn_varlen_fwd(q, k, k, plan, o=o, lse=lse)
    assert (o == 7).all() and (lse == 7).all()
    plan = A.attn_varlen_plan(ints([0, 0]), 0, H, Hkv)
    o, lse = A.attn_varlen_fwd(q[:0], k[:0], k[:0], plan)
    assert o.shape == (0, H, d) and lse.shape == (0, H)
    c = Cache(4, Hkv, 16, d, [[0, 1]])
    A.attn_cache_append_int8(k[:0], k[:0], *c.gpu, ints([0, 0]), ints([3]))
    x, _ = A.attn_cache_read_int8(*c.gpu, ints([0, 0]), ints([3]), 0)
    assert x.shape == (0, Hkv, d) and c.equal()
    for width in (2, 200):  # whole sequences, and split ones
        c = Cache(4, Hkv, 16, d, [[], []], width=width)
        o, lse = A.attn_decode_int8(normal((2, 3, H, d), 1).cuda(), *c.gpu, ints([0, 0]))
        assert (o == 0).all() and (lse == -torch.inf).all()
    A.attn_check_status()


def test_two_streams_at_once(A):
    """Calls of every kind overlap on two streams, each with its own workspace and outputs."""
    H, Hkv, d, page, lens = 8, 2, 128, 64, [3000, 70, 900]
    T, cu = 1500, [0, 700, 1500]
    tables, pages = scattered([-(-n // page) for n in lens], 5)
    c = Cache(pages, Hkv, page, d, tables)
    q = normal((3, 1, H, d), 1).cuda()
    x = normal((T, H + 2 * Hkv, d), 2).cuda()
    L, cus, zero = ints(lens), ints(cu), ints([0, 0])
    scratch = [Cache(30, Hkv, page, d, [list(range(14)), list(range(14, 28))], seed=i).gpu for i in range(2)]

    def run(i):
        plan = A.attn_varlen_plan(cus, T, H, Hkv)
        out = []
        for _ in range(6):
            out += A.attn_varlen_fwd(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], plan)
            out += A.attn_decode_int8(q, *c.gpu, L)
            A.attn_cache_append_int8(x[:, H:H + Hkv], x[:, H + Hkv:], *scratch[i], cus, zero)
            out += A.attn_cache_read_int8(*scratch[i], cus, zero, T)
        return out

    want = run(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got.append(run(i))
    A.attn_check_status(streams[0])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
