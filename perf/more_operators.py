"""Workloads of the serving operators around the paged INT8 cache: block tables
and slot maps built on the GPU from the requests' lengths, and the attention of
a batch whose sequences share a long prefix.

`run` computes them in plain torch operations, or, where `own` is true, with
the framework's calls.  Two kinds of case:

  reserve  a step's pages are taken from the stack of free pages (requests that
           end give theirs back first), with the offsets, slots and positions of
           the new tokens; then the step is taken back, as drafted tokens that
           were rejected are, which leaves table and stack as they were.
  shared   the newest `new` tokens of every sequence attend over a prefix that
           all of them share, stored once, and over their own pages; outputs O and
           the log-sum-exp.

The lengths of a case's sequences follow from the case alone (`spread` is their
seed): the first is `longest`, the others lie between `shortest` and `longest`,
uniformly in their logarithm.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # A decoding step of a small batch: latency counts.
        dict(name="reserve-step", kind="reserve", seqs=3, longest=1, shortest=1, held=700, ends=0.0, room=2.0, page=16,
             spread=0),
        # A decoding step of a large batch in which some requests end.
        dict(name="reserve-step-batch", kind="reserve", seqs=256, longest=1, shortest=1, held=3000, ends=0.1, room=1.5,
             page=64, spread=1),
        # Prompts, or further parts of prompts, admitted at once.
        dict(name="reserve-prompts", kind="reserve", seqs=64, longest=4096, shortest=150, held=2000, ends=0.2, room=1.2,
             page=64, spread=2),
        # A thousand ragged prompts in small pages, more than there are pages for.
        dict(name="reserve-scarce", kind="reserve", seqs=1000, longest=6000, shortest=10, held=1000, ends=0.1, room=0.8,
             page=16, spread=3),
        # Two short questions behind a short instruction to a small model: latency counts.
        dict(name="shared-two-short", kind="shared", prefix=300, seqs=2, longest=24, shortest=3, new=1, heads=8,
             kv_heads=2, dim=64, page=16, spread=4),
        # Four samples of the answer to one long document: the prefix's bytes.
        dict(name="shared-four-long", kind="shared", prefix=100003, seqs=4, longest=700, shortest=90, new=1, heads=32,
             kv_heads=8, dim=128, page=64, spread=5),
        # A served batch behind one long instruction.
        dict(name="shared-batch", kind="shared", prefix=16000, seqs=64, longest=1500, shortest=20, new=1, heads=32,
             kv_heads=8, dim=128, page=64, spread=6),
        # Ungrouped heads of 64 and small pages.
        dict(name="shared-h12-d64", kind="shared", prefix=9001, seqs=48, longest=800, shortest=30, new=1, heads=12,
             kv_heads=12, dim=64, page=16, spread=7),
        # Drafted tokens checked at once: five query tokens each, pages of 32.
        dict(name="shared-drafted", kind="shared", prefix=5000, seqs=24, longest=400, shortest=9, new=5, heads=32,
             kv_heads=8, dim=128, page=32, spread=8),
        # Seven query heads a key head, two key heads, pages of 128.
        dict(name="shared-group-of-7", kind="shared", prefix=30000, seqs=40, longest=500, shortest=40, new=1, heads=14,
             kv_heads=2, dim=128, page=128, spread=9),
        # Questions of a hundred tokens read behind one document.
        dict(name="shared-questions", kind="shared", prefix=12000, seqs=16, longest=400, shortest=100, new=100, heads=32,
             kv_heads=8, dim=128, page=64, spread=10),
        # Many samples at once behind a long prefix.
        dict(name="shared-large-batch", kind="shared", prefix=32768, seqs=256, longest=1000, shortest=50, new=1,
             heads=32, kv_heads=8, dim=128, page=64, spread=11),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1 << 30)
    if rng.random() < 0.3:
        longest = rng.choice([1, _log_uniform(rng, 1, 6000)])
        seqs = _log_uniform(rng, 1, max(1, min(1000, 1200000 // longest)))
        return dict(kind="reserve", seqs=seqs, longest=longest, shortest=_log_uniform(rng, 1, longest),
                    held=_log_uniform(rng, 1, 4000), ends=rng.choice([0.0, 0.1, 0.5]), room=rng.choice([0.6, 1.0, 2.0]),
                    page=page, spread=spread)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    heads = kv_heads * group
    new = rng.choice([1, 1, 1, 2, 3, 5, 8, _log_uniform(rng, 9, 128)])
    prefix = _log_uniform(rng, 1, 131072)
    longest = _log_uniform(rng, new, max(new, 3000))
    # The scores stay below those of the largest listed case, and so does the work.
    most = int(2.4e8 / (heads * new * (prefix + longest)))
    seqs = _log_uniform(rng, 1, max(1, min(200, most)))
    return dict(kind="shared", prefix=prefix, seqs=seqs, longest=longest, shortest=_log_uniform(rng, new, longest),
                new=new, heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]), page=page, spread=spread)


def _lengths(case):
    rng = random.Random(case["spread"])
    return [case["longest"]] + [_log_uniform(rng, case["shortest"], case["longest"]) for _ in range(case["seqs"] - 1)]


def _step(case):
    """Positions that the sequences of a reserve case hold before and after the step: some are new, some go on, some
    end."""
    rng = random.Random(case["spread"] + 1)
    held, wanted = [], []
    for n in _lengths(case):
        a = 0 if rng.random() < 0.2 else rng.randint(0, case["held"])
        held.append(a)
        wanted.append(0 if a and rng.random() < case["ends"] else a + n)
    return held, wanted


def _pages(n, page):
    return -(-n // page)


def _served(case):
    """(free pages before the step, positions after it): the requests are served in their order while pages are left."""
    held, wanted = _step(case)
    page = case["page"]
    need = [max(0, _pages(w, page) - _pages(a, page)) for a, w in zip(held, wanted)]
    back = sum(max(0, _pages(a, page) - _pages(w, page)) for a, w in zip(held, wanted))
    free = max(0, int(case["room"] * sum(need)) - back)
    after, upto = [], 0
    for a, w, n in zip(held, wanted, need):
        upto += n
        after.append(w if n == 0 or upto <= free + back else a)
    return free, after


def _new(before, after):
    return sum(max(0, y - x) for x, y in zip(before, after))


# --------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _table(pages_of, order, width):
    """Rows of page numbers taken from `order` one behind the other, -1 behind them."""
    rows, at = [], 0
    for n in pages_of:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return _ints(rows)


def _pool(pages, case, g):
    """Pages as they are after writing values of different size from channel to channel: (codes, scales)."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    size = torch.exp(0.5 * _normal((h, 1, d), g))
    codes = torch.empty((pages, h, p, d), dtype=torch.int8, device=DEVICE)
    scales = torch.empty((pages, h), dtype=torch.float32, device=DEVICE)
    for at in range(0, pages, 4096):  # in parts, for the memory's sake
        x = (_normal((min(4096, pages - at), h, p, d), g) * size).bfloat16().float()
        s = (x.abs().amax((2, 3)).double() / 127).float()
        scales[at:at + len(x)] = s
        codes[at:at + len(x)] = torch.round(x / s[:, :, None, None]).clamp_(-127, 127).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    g, g_cpu = _generator(seed), torch.Generator().manual_seed(int(seed))
    page, st = case["page"], {"case": case}
    if case["kind"] == "reserve":
        held, wanted = _step(case)
        free, after = _served(case)
        used = [_pages(a, page) for a in held]
        total = free + sum(used)
        order = torch.randperm(total + 1, generator=g_cpu).tolist()
        st["table"] = _table(used, order, max(1, max(_pages(max(x), page) for x in zip(held, wanted))))
        st["stack"] = _ints(order[sum(used):sum(used) + free] + [-1] * (total + 1 - free))
        st["free"] = _ints([free])
        st["held"], st["wanted"] = _ints(held), _ints(wanted)
        # What the host knows: the rows that it has packed for the step, and room for those that come back.
        st["tokens"], st["tokens_back"] = max(1, _new(held, wanted)), max(1, _new(after, held))
        return st
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    own_pages = [_pages(n, page) for n in lengths]
    prefix_pages = _pages(case["prefix"], page)
    total = prefix_pages + sum(own_pages)
    order = torch.randperm(total + 3, generator=g_cpu)[:total].tolist()
    st["q"] = _normal((case["seqs"], case["new"], h, d), g).bfloat16()
    st["prefix_table"] = _ints(order[:prefix_pages])
    st["prefix_len"] = _ints([case["prefix"]])
    st["table"] = _table(own_pages, order[prefix_pages:], max(own_pages))
    st["seqlens"] = _ints(lengths)
    st["k_cache"], st["k_scale"] = _pool(total + 3, case, g)
    st["v_cache"], st["v_scale"] = _pool(total + 3, case, g)
    if own:
        # Allocated once, as every step of a batch of this size uses it.
        import precision_numerics_gb300 as pn
        st["workspace"] = torch.empty(
            max(1, pn.attn_decode_shared_int8_workspace_bytes(case["seqs"], case["new"], h, hk, d, page, prefix_pages,
                                                              st["table"].shape[1])), dtype=torch.uint8, device=DEVICE)
    return st


# ----------------------------------------------------------------------- runs
def run(st):
    if st["case"]["kind"] == "reserve":
        reserve = _reserve
        if own:
            import precision_numerics_gb300 as pn
            reserve = pn.attn_cache_reserve
        step = reserve(st["table"], st["held"], st["wanted"], st["stack"], st["free"], st["case"]["page"], st["tokens"])
        back = reserve(st["table"], step[0], st["held"], st["stack"], st["free"], st["case"]["page"], st["tokens_back"])
        return (*step, *back, st["table"], st["stack"], st["free"])
    if own:
        import precision_numerics_gb300 as pn
        return pn.attn_decode_shared_int8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                          st["prefix_table"], st["prefix_len"], st["table"], st["seqlens"],
                                          workspace=st["workspace"])
    return _shared(st)


def _reserve(table, held, wanted, stack, free, page, tokens):
    """Moves the pages between table and stack; returns the lengths afterwards, the new tokens' offsets, and each one's
    row in the pool of pages and position."""
    dev, width = table.device, table.shape[1]
    held, wanted = held.long(), wanted.long()
    have, want = (held + page - 1) // page, (wanted + page - 1) // page
    need = (want - have).clamp(min=0)
    j = torch.arange(width, device=dev)[None]
    # Released pages go on top of the stack.  One place more takes what is not meant.
    gone = (j >= want[:, None]) & (j < have[:, None])
    at = free + torch.cumsum(gone.view(-1), 0).view(gone.shape) - 1
    room = torch.cat([stack, stack[:1]])
    room[torch.where(gone, at, torch.full_like(at, len(stack)))] = table
    stack.copy_(room[:-1])
    top = free.long() + gone.sum()
    # The pages of all requests that are served are the top ones.
    upto = torch.cumsum(need, 0)
    served = (need == 0) | (upto <= top)
    top = top - (need * served).sum()
    fresh = (j >= have[:, None]) & (j < want[:, None])
    taken = fresh & served[:, None]
    at = (top + torch.cumsum(taken.view(-1), 0).view(taken.shape) - 1).clamp(min=0)
    table.copy_(torch.where(taken, stack[at], torch.where(gone | fresh, torch.full_like(table, -1), table)))
    free.copy_(top)
    cu = torch.zeros(len(held) + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.cumsum((wanted - held).clamp(min=0), 0)
    t = torch.arange(tokens, device=dev)
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=len(held) - 1)
    inside = t < cu[-1]
    pos = torch.where(inside, t - cu[seq] + held[seq], torch.zeros_like(t))
    pages = table[seq, pos // page].long()
    slots = torch.where(inside & served[seq], pages * page + pos % page, torch.full_like(t, -1))
    pos = torch.where(inside, pos, torch.full_like(t, -1))
    return torch.where(served, wanted, held).int(), cu.int(), slots.int(), pos.int()


def _shared(st):
    """Prefix and own histories apart; their maxima and sums are joined before the division."""
    case, b, m, h, d = st["case"], *st["q"].shape
    hk, page = case["kv_heads"], case["page"]
    group = h // hk

    def values(ids, n):  # [..., pages] -> [..., hk, n, d]
        k = st["k_cache"][ids].float() * st["k_scale"][ids][..., None, None]
        v = st["v_cache"][ids].float() * st["v_scale"][ids][..., None, None]
        shape = (*ids.shape[:-1], hk, n, d)
        return k.transpose(-4, -3).reshape(shape), v.transpose(-4, -3).reshape(shape)

    pre, table = st["prefix_table"].long(), st["table"].long().clamp(min=0)
    n0, n1 = pre.shape[0] * page, table.shape[1] * page
    q = st["q"].float().view(b, m, hk, group, d).permute(2, 0, 1, 3, 4)  # [hk, b, m, group, d]
    k, v = values(pre, n0)
    s0 = torch.matmul(q.reshape(hk, -1, d), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(hk, b, m, group, n0)
    s0.masked_fill_(torch.arange(n0, device=q.device) >= st["prefix_len"], float("-inf"))
    k1, v1 = values(table, n1)
    q1 = q.transpose(0, 1).reshape(b, hk, m * group, d)
    s1 = torch.matmul(q1, k1.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(b, hk, m, group, n1)
    last = st["seqlens"].long()[:, None] - m + torch.arange(m, device=q.device)  # [b, m]: the last own key a token sees
    hidden = torch.arange(n1, device=q.device) > last[..., None]
    s1 = s1.masked_fill(hidden[:, None, :, None], float("-inf")).transpose(0, 1)  # [hk, b, m, group, n1]
    top = torch.maximum(s0.amax(-1), s1.amax(-1)).clamp(min=torch.finfo(torch.float32).min)[..., None]
    p0, p1 = torch.exp(s0.sub_(top)), torch.exp(s1 - top)
    total = p0.sum(-1, keepdim=True) + p1.sum(-1, keepdim=True)
    o = torch.matmul(p0.view(hk, -1, n0), v).view(hk, b, m, group, d)
    o = o + torch.matmul(p1.transpose(0, 1).reshape(b, hk, -1, n1), v1).view(b, hk, m, group, d).transpose(0, 1)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    return o.permute(1, 2, 0, 3, 4).reshape(b, m, h, d).bfloat16(), lse.permute(1, 2, 0, 3).reshape(b, m, h)


# ----------------------------------------------------------------------- work
def work(case):
    page = case["page"]
    if case["kind"] == "reserve":
        held, wanted = _step(case)
        _, after = _served(case)
        total = 0
        for x, want, y in ((held, wanted, after), (after, held, held)):
            moved = sum(abs(_pages(b, page) - _pages(a, page)) for a, b in zip(x, y))
            fresh = [max(0, b - a) for a, b in zip(x, want)]
            begun = sum(1 for a, b in zip(x, want) if b > a and a % page)
            # Lengths in and out, offsets; a number out of one place into another; pages begun earlier; slots and
            # positions.
            total += 4 * (4 * len(x) + 1) + 8 * moved + 4 * begun + 8 * sum(fresh) + 8
        return {"bytes": total, "flops": 0}
    h, hk, d, m = case["heads"], case["kv_heads"], case["dim"], case["new"]
    lengths, n0 = _lengths(case), case["prefix"]
    pages = _pages(n0, page) + sum(_pages(n, page) for n in lengths)
    pairs = sum(n0 + max(0, n - m + 1 + i) for n in lengths for i in range(m))
    return {"bytes": 2 * hk * d * (n0 + sum(lengths)) + 8 * hk * pages + 4 * pages + len(lengths) * m * h * (4 * d + 4),
            "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------- exact
def _exact_reserve(table, held, wanted, stack, page, tokens):
    """One request after the other, on lists; stack is (numbers, how many of them are free)."""
    numbers, free = stack
    for b, (a, w) in enumerate(zip(held, wanted)):
        for j in range(_pages(w, page), _pages(a, page)):
            numbers[free] = table[b][j]
            table[b][j] = -1
            free += 1
    lens, asked, taken = [], 0, 0
    for a, w in zip(held, wanted):
        need = max(0, _pages(w, page) - _pages(a, page))
        asked += need
        fits = need == 0 or asked <= free
        taken += need if fits else 0
        lens.append(w if fits else a)
    free -= taken
    cu, slots, positions, at = [0], [], [], free
    for b, (a, w) in enumerate(zip(held, wanted)):
        for j in range(_pages(a, page), _pages(w, page)):
            table[b][j] = numbers[at] if lens[b] == w else -1
            at += 1 if lens[b] == w else 0
        for pos in range(a, w):
            slots.append(table[b][pos // page] * page + pos % page if lens[b] == w else -1)
            positions.append(pos)
        cu.append(len(positions))
    none = [-1] * (tokens - len(slots))
    return (lens, cu, slots + none, positions + none), (numbers, free)


def exact(case, seed):
    st = prepare(case, seed)
    page = case["page"]
    if case["kind"] == "reserve":
        table, held, wanted = st["table"].tolist(), st["held"].tolist(), st["wanted"].tolist()
        stack = (st["stack"].tolist(), st["free"].item())
        step, stack = _exact_reserve(table, held, wanted, stack, page, st["tokens"])
        back, stack = _exact_reserve(table, step[0], held, stack, page, st["tokens_back"])
        return (*map(_ints, step), *map(_ints, back), _ints(table), _ints(stack[0]), _ints([stack[1]]))
    lengths, hk, d, n0 = _lengths(case), case["kv_heads"], case["dim"], case["prefix"]
    b, m, h = st["q"].shape[:3]
    group = h // hk
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros((b, m, h), dtype=torch.float64, device=DEVICE)

    def rows(codes, scales, ids, c, n):
        return (codes[ids, c].double() * scales[ids, c].double()[:, None, None]).view(-1, d)[:n]

    pre = st["prefix_table"].long()
    at_once = max(1, (1 << 28) // (m * group * (n0 + max(lengths))))  # sequences whose scores are held together
    for c in range(hk):
        heads = slice(c * group, (c + 1) * group)
        k0 = rows(st["k_cache"], st["k_scale"], pre, c, n0)
        v0 = rows(st["v_cache"], st["v_scale"], pre, c, n0)
        for first in range(0, b, at_once):
            some = range(first, min(b, first + at_once))
            q = st["q"][first:first + at_once, :, heads].double()
            s0 = (q.reshape(-1, d) @ k0.t() / math.sqrt(d)).view(len(some), m * group, n0)
            lse0 = torch.logsumexp(s0, -1)
            o0 = (torch.exp(s0 - lse0[..., None]).view(-1, n0) @ v0).view(len(some), m * group, d)
            for i in some:
                n = lengths[i]
                ids = st["table"][i, :_pages(n, page)].long()
                k1 = rows(st["k_cache"], st["k_scale"], ids, c, n)
                v1 = rows(st["v_cache"], st["v_scale"], ids, c, n)
                s1 = q[i - first].reshape(-1, d) @ k1.t() / math.sqrt(d)
                last = torch.arange(n - m, n, device=DEVICE).repeat_interleave(group)
                s1[torch.arange(n, device=DEVICE)[None] > last[:, None]] = -math.inf
                both = torch.logaddexp(lse0[i - first], torch.logsumexp(s1, -1))
                part = torch.exp(s1 - both[:, None]) @ v1 + torch.exp(lse0[i - first] - both)[:, None] * o0[i - first]
                o[i, :, heads], lse[i, :, heads] = part.view(m, group, d), both.view(m, group)
    return o, lse
