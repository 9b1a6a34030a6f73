"""Steps in which pages run out: the rows of requests that were not served leave the cache as it was."""
import math

import pytest

import serving_ref as ref
from test_serving_gpu import A, BF, Cache, ints, normal, scattered, sums  # noqa: F401
from test_shared_gpu import check

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("many", [False, True])
def test_append_up_to_lens(A, many, page, d, monkeypatch):
    """No rows of a sequence, some, all, and lens behind the last; a step's few rows a sequence and prompts, whose
    kernels differ.  Rows that are left out have no page and would make every scale grow."""
    from precision_numerics_gb300 import attn

    Hkv, more = 3, 2 * page if many else 0
    starts = [0, 5, page - 1, page, 3 * page + 2, 7, 2, 0]
    lens = [n + (more if n else 0) for n in (1, 1, 2, 3, 3, 0, 4, 3)]
    kept = [0, 0, 1, 2, lens[4], 0, 2, 3]
    ends = [s + n for s, n in zip(starts, kept)]
    ends[4] += 100
    ends[7] += 2 ** 31 - 4  # 2^31 - 1
    kept[7] = lens[7]
    ends[5] = 0  # held less than it held: nothing new, nothing lost
    T, cu = sum(lens), sums(lens)
    assert (T <= 8 * len(lens)) != many
    tables, pages = scattered([-(-(s + n) // page) for s, n in zip(starts, kept)], 1)
    c = Cache(pages, Hkv, page, d, tables)
    rows = [normal((T, Hkv, d), 1), normal((T, Hkv, d), 2) * 0.01]
    out = [cu[b] + i for b in range(len(lens)) for i in range(kept[b], lens[b])]
    for x in rows:
        x[out] *= 2.0 ** 30
    for i in range(2):
        for b, t in enumerate(c.tables):
            ref.append(rows[i][cu[b]:cu[b] + kept[b]], c.codes[i], c.scales[i], t, starts[b])
    args = (rows[0].cuda(), rows[1].cuda(), *c.gpu, ints(cu), ints(starts))
    A.attn_cache_append_int8(*args, lens=ints(ends))
    A.attn_check_status()
    assert c.equal()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    A.attn_cache_append_int8(*args, stream=side, lens=ints(ends))
    monkeypatch.setattr(attn, "_BINDING", attn._NoBinding)
    A.attn_cache_append_int8(*args, lens=ints(ends))
    A.attn_check_status()
    assert c.equal()
    # A length below 0 leaves its sequence out, and is reported.
    fresh = Cache(pages, Hkv, page, d, tables)
    for i in range(2):
        for b, t in enumerate(fresh.tables):
            if b != 3:
                ref.append(rows[i][cu[b]:cu[b] + kept[b]], fresh.codes[i], fresh.scales[i], t, starts[b])
    gpu = Cache(pages, Hkv, page, d, tables).gpu
    A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *gpu, *args[-2:], lens=ints(ends[:3] + [-1] + ends[4:]))
    with pytest.raises(A.AttnError, match="out of range"):
        A.attn_check_status()
    fresh.gpu = gpu
    assert fresh.equal()


@pytest.mark.parametrize("rows_each", [3, 40])
def test_append_up_to_lens_many_sequences(A, rows_each):
    """More sequences than threads look for the pages at a time; a third of them is left out."""
    B, Hkv, page, d = 700, 2, 16, 64
    g = torch.Generator().manual_seed(3)
    starts = torch.randint(0, 50, (B,), generator=g).tolist()
    lens = torch.randint(0, rows_each, (B,), generator=g).tolist()
    kept = [0 if b % 3 == 1 else n for b, n in enumerate(lens)]
    T, cu = sum(lens), sums(lens)
    assert (T <= 8 * B) == (rows_each == 3)
    tables, pages = scattered([-(-(s + n) // page) for s, n in zip(starts, kept)], 2)
    c = Cache(pages, Hkv, page, d, tables, width=6)
    rows = [normal((T, Hkv, d), 1), normal((T, Hkv, d), 2)]
    for i in range(2):
        for b, t in enumerate(c.tables):
            ref.append(rows[i][cu[b]:cu[b] + kept[b]], c.codes[i], c.scales[i], t, starts[b])
    A.attn_cache_append_int8(rows[0].cuda(), rows[1].cuda(), *c.gpu, ints(cu), ints(starts),
                             lens=ints([s + n for s, n in zip(starts, kept)]))
    A.attn_check_status()
    assert c.equal()


def test_append_up_to_lens_refuses(A):
    c = Cache(4, 2, 16, 64, [[0], [1]])
    x, cu, starts = normal((4, 2, 64), 1).cuda(), ints([0, 2, 4]), ints([0, 0])
    for lens in (ints([1]), ints([1, 1]).long(), ints([1, 1]).cpu(), ints([1, 1])[:, None]):
        with pytest.raises(ValueError, match="lens"):
            A.attn_cache_append_int8(x, x, *c.gpu, cu, starts, lens=lens)
    with pytest.raises(TypeError, match="lens"):
        A.attn_cache_append_int8(x, x, *c.gpu, cu, starts, lens=[1, 1])
    lib, args = A.load_library(), [t.data_ptr() for t in (*c.gpu, cu, starts)]
    good = ints([1, 1]).data_ptr()
    for lens, word, T in ((None, "lens", 4), (good + 2, "lens", 4), (None, "lens", 0), (good, "", 0)):
        status = lib.attn_cache_append_served_int8(x.data_ptr(), x.data_ptr(), 128, 64, 128, 64, *args, lens, 2, T, 2, 64, 4,
                                                   16, 1, None)
        assert (status == A.ATTN_ERR_INVALID_ARG and word in lib.attn_last_error().decode()) if word else status == 0
    A.attn_check_status()
    assert c.equal()


@pytest.mark.parametrize("shared", [False, True])
def test_steps_that_run_out_of_pages(A, shared):
    """A captured step of reserve, append and attend, replayed while pages run out: whoever is not served keeps its codes
    and scales, nothing is reported, and it goes on in a later step when another request has ended."""
    H, Hkv, d, page, n_q, B, width, pages, n0 = 8, 2, 64, 16, 3, 5, 8, 18, 20
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()
    pre, free = order[:2], order[2:]
    c = Cache(pages, Hkv, page, d, [[] for _ in range(B)], width=width)
    table, stack, n_free = c.gpu[4], ints(free + [-1, -1]), ints([len(free)])
    table_list, stack_list, free_count = [[-1] * width for _ in range(B)], free + [-1, -1], len(free)
    T = B * n_q
    rows = torch.zeros((B, n_q, H + 2 * Hkv, d), dtype=BF, device="cuda")
    held, wanted, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    o, lse = torch.zeros((B, n_q, H, d), dtype=BF, device="cuda"), torch.zeros((B, n_q, H), device="cuda")
    need = (A.attn_decode_shared_int8_workspace_bytes(B, n_q, H, Hkv, d, page, len(pre), width) if shared
            else A.attn_decode_int8_workspace_bytes(B, n_q, H, Hkv, d, page, width))
    ws, prefix, prefix_len = torch.empty(need + 1, dtype=torch.uint8, device="cuda"), ints(pre), ints([n0])
    slots, positions = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))

    def step():
        A.attn_cache_reserve(table, held, wanted, stack, n_free, page, T, lens=lens, cu_seqlens=cu, slots=slots,
                             positions=positions)
        flat = rows.view(T, H + 2 * Hkv, d)
        A.attn_cache_append_int8(flat[:, H:H + Hkv], flat[:, H + Hkv:], *c.gpu, cu, held, lens=lens)
        if shared:
            A.attn_decode_shared_int8(rows[:, :, :H], *c.gpu[:4], prefix, prefix_len, table, lens, o=o, lse=lse,
                                      workspace=ws)
        else:
            A.attn_decode_int8(rows[:, :, :H], *c.gpu, lens, o=o, lse=lse, workspace=ws)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    have, waited, went_on = [0, 0, 0, 0, 0], set(), set()
    for s in range(40):
        x = normal((B, n_q, H + 2 * Hkv, d), 20 + s) * (1 + s)  # scales grow with every step
        rows.copy_(x)
        want = [n + n_q for n in have]
        if s % 13 == 12:  # the longest ends
            want[have.index(max(have))] = 0
        want = [min(w, width * page) for w in want]
        held.copy_(ints(have))
        wanted.copy_(ints(want))
        graph.replay()
        A.attn_check_status()
        after, offsets, _, _, free_count = ref.reserve(table_list, have, want, stack_list, free_count, page, T, pages)
        assert lens.tolist() == after and cu.tolist() == offsets and table.tolist() == table_list
        flat = x.view(T, H + 2 * Hkv, d)
        c.tables = [[p for p in t if p >= 0] for t in table_list]
        for b in range(B):
            n = max(after[b] - have[b], 0)
            for i, part in enumerate((flat[:, H:H + Hkv], flat[:, H + Hkv:])):
                ref.append(part[offsets[b]:offsets[b] + n], c.codes[i], c.scales[i], c.tables[b], have[b])
            if after[b] < want[b]:
                waited.add(b)
            elif b in waited and want[b] > have[b]:
                went_on.add(b)
        assert c.equal()
        check(c, pre if shared else [], n0 if shared else 0, x[:, :, :H], after, 1 / math.sqrt(d), o, lse)
        have = after
    assert waited and went_on
