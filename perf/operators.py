"""Workloads of the serving operators: prompt attention over packed sequences,
writing to and reading from a paged INT8 cache of keys and values, and the
attention of the newest tokens over that cache.

`run` computes them in plain torch operations, or, where `own` is true, with
the framework's calls.  Three kinds of case:

  prompt  attention over whole prompts packed one behind the other, grouped
          heads; outputs O and the log-sum-exp.
  write   new keys and values go into their sequences' pages (one scale per
          page and head; a page that was begun earlier keeps what it holds),
          then the touched pages' values are read back.
  decode  the newest `new` tokens of every sequence attend over the cache;
          outputs O and the log-sum-exp.

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
        # A short question to a small model: one sequence, latency counts.
        dict(name="prompt-one-short", kind="prompt", seqs=1, longest=23, shortest=23, heads=8, kv_heads=2, dim=64,
             causal=True, fused=False, spread=0),
        # A batch of ragged prompts with four query heads per key head; q, k and v are views of one projection's output.
        dict(name="prompt-ragged-grouped", kind="prompt", seqs=12, longest=2048, shortest=65, heads=32, kv_heads=8,
             dim=128, causal=True, fused=True, spread=1),
        # Ungrouped heads of 64, the shape of the repository's smaller causal workload with ragged lengths.
        dict(name="prompt-ragged-h12-d64", kind="prompt", seqs=8, longest=1024, shortest=200, heads=12, kv_heads=12,
             dim=64, causal=True, fused=False, spread=2),
        # Documents embedded without a causal mask.
        dict(name="prompt-full-mask", kind="prompt", seqs=10, longest=1500, shortest=31, heads=16, kv_heads=4, dim=128,
             causal=False, fused=False, spread=3),
        # One long document.
        dict(name="prompt-long", kind="prompt", seqs=1, longest=16384, shortest=16384, heads=16, kv_heads=2, dim=128,
             causal=True, fused=False, spread=4),
        # A decoding step of a small batch: one token each goes into a page begun earlier.
        dict(name="write-step", kind="write", seqs=3, longest=1, shortest=1, held=700, kv_heads=4, dim=64, page=16,
             spread=5),
        # A decoding step of a large batch.
        dict(name="write-step-batch", kind="write", seqs=96, longest=1, shortest=1, held=3000, kv_heads=8, dim=128,
             page=64, spread=6),
        # Prompts, or further parts of prompts, written at once.
        dict(name="write-prompts", kind="write", seqs=16, longest=4096, shortest=150, held=2000, kv_heads=8, dim=128,
             page=64, spread=7),
        # One user, a short history: latency counts.
        dict(name="decode-one-short", kind="decode", seqs=1, longest=77, shortest=77, new=1, heads=8, kv_heads=2, dim=64,
             page=16, spread=8),
        # One user, a long history: few rows, the work is split along the keys.
        dict(name="decode-one-long", kind="decode", seqs=1, longest=131000, shortest=131000, new=1, heads=32, kv_heads=8,
             dim=128, page=64, spread=9),
        # A served batch of ragged histories; the largest.
        dict(name="decode-batch", kind="decode", seqs=64, longest=16000, shortest=500, new=1, heads=32, kv_heads=8,
             dim=128, page=64, spread=10),
        # Drafted tokens checked at once: five query tokens each, pages of 32.
        dict(name="decode-drafted", kind="decode", seqs=24, longest=5000, shortest=100, new=5, heads=32, kv_heads=8,
             dim=128, page=32, spread=11),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prompt", "write", "decode"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    spread = rng.randrange(1 << 30)
    if kind == "prompt":
        longest = _log_uniform(rng, 1, 8192)
        # The plain form's scores stay below about 16 GB and the work below the largest listed case's.
        most = max(1, min(48, int(3.5e9 / (kv_heads * group * longest * longest))))
        return dict(kind=kind, seqs=_log_uniform(rng, 1, most), longest=longest, shortest=_log_uniform(rng, 1, longest),
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, causal=rng.random() < 0.75,
                    fused=rng.random() < 0.5, spread=spread)
    page = rng.choice([16, 32, 64, 128])
    if kind == "write":
        longest = rng.choice([1, _log_uniform(rng, 1, 6000)])
        seqs = _log_uniform(rng, 1, max(1, min(128, 60000 // longest)))
        return dict(kind=kind, seqs=seqs, longest=longest, shortest=_log_uniform(rng, 1, longest),
                    held=_log_uniform(rng, 1, 4000), kv_heads=kv_heads, dim=dim, page=page, spread=spread)
    new = rng.choice([1, 1, 1, 2, 3, 4, 6, 8])
    longest = _log_uniform(rng, new, 131072)
    seqs = _log_uniform(rng, 1, max(1, min(128, 900000 // (longest * kv_heads))))
    return dict(kind=kind, seqs=seqs, longest=longest, shortest=_log_uniform(rng, min(new, longest), longest), new=new,
                heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, spread=spread)


def _lengths(case):
    rng = random.Random(case["spread"])
    return [case["longest"]] + [_log_uniform(rng, case["shortest"], case["longest"]) for _ in range(case["seqs"] - 1)]


def _held(case):
    """Tokens that each sequence of a write case holds already: some begin, some go on."""
    rng = random.Random(case["spread"] + 1)
    return [0 if rng.random() < 0.2 else rng.randint(0, case["held"]) for _ in range(case["seqs"])]


def _sums(lengths):
    total = [0]
    for n in lengths:
        total.append(total[-1] + n)
    return total


# --------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _block_table(pages_of, g_cpu):
    """A table of scattered pages: row b lists sequence b's, -1 behind them.  Also the number of pages of the pool."""
    total = sum(pages_of)
    order = torch.randperm(total + 3, generator=g_cpu)[:total].tolist()
    width = max(max(pages_of), 1)
    rows, at = [], 0
    for n in pages_of:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return _ints(rows), total + 4  # the last page is nobody's


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
    h, hk, d = case.get("heads"), case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    st = {"case": case, "lengths": lengths}
    if case["kind"] == "prompt":
        t = sum(lengths)
        if case["fused"]:
            rows = _normal((t, h + 2 * hk, d), g).bfloat16()
            st["q"], st["k"], st["v"] = rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:]
        else:
            st["q"], st["k"], st["v"] = (_normal((t, n, d), g).bfloat16() for n in (h, hk, hk))
        st["cu_seqlens"] = _ints(_sums(lengths))
        if own:
            # Made once for a batch of prompts; every layer of a model uses it.
            import precision_numerics_gb300 as pn
            st["plan"] = pn.attn_varlen_plan(st["cu_seqlens"], t, h, hk, causal=case["causal"])
        return st
    page = case["page"]
    if case["kind"] == "write":
        held = _held(case)
        ends = [a + n for a, n in zip(held, lengths)]
        first = [a // page * page for a in held]  # where the touched pages begin
        t = sum(lengths)
        st["k"] = (_normal((t, hk, d), g) * torch.exp(0.7 * _normal((t, 1, 1), g))).bfloat16()
        st["v"] = _normal((t, hk, d), g).bfloat16()
        st["cu_seqlens"], st["starts"] = _ints(_sums(lengths)), _ints(held)
        back = [e - f for e, f in zip(ends, first)]
        st["read_total"], st["read_most"] = sum(back), max(back)
        st["read_cu"], st["read_starts"] = _ints(_sums(back)), _ints(first)
        st["table"], pages = _block_table([-(-e // page) for e in ends], g_cpu)
        st["touched"] = max(-(-e // page) - f // page for e, f in zip(ends, first))
    else:
        st["q"] = _normal((case["seqs"], case["new"], h, d), g).bfloat16()
        st["seqlens"] = _ints(lengths)
        st["table"], pages = _block_table([-(-n // page) for n in lengths], g_cpu)
        if own:
            import precision_numerics_gb300 as pn
            st["workspace"] = torch.empty(
                max(1, pn.attn_decode_int8_workspace_bytes(case["seqs"], case["new"], h, hk, d, page,
                                                           st["table"].shape[1])), dtype=torch.uint8, device=DEVICE)
    st["k_cache"], st["k_scale"] = _pool(pages, case, g)
    st["v_cache"], st["v_scale"] = _pool(pages, case, g)
    return st


# ----------------------------------------------------------------------- runs
def run(st):
    kind = st["case"]["kind"]
    if own:
        import precision_numerics_gb300 as pn
        if kind == "prompt":
            return pn.attn_varlen_fwd(st["q"], st["k"], st["v"], st["plan"], causal=st["case"]["causal"])
        cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"])
        if kind == "write":
            pn.attn_cache_append_int8(st["k"], st["v"], *cache, st["cu_seqlens"], st["starts"])
            k, v = pn.attn_cache_read_int8(*cache, st["read_cu"], st["read_starts"], st["read_total"],
                                           dtype=torch.float32)
            return k, v, st["k_scale"], st["v_scale"]
        return pn.attn_decode_int8(st["q"], *cache, st["seqlens"], workspace=st["workspace"])
    if kind == "prompt":
        return _prompt(st)
    if kind == "write":
        return _write(st)
    return _decode(st)


def _softmax_v(s, v, visible):
    """Rows of softmax(s) v over the visible keys, and the log-sum-exp: s [..., m, n], v [..., n, d] in 32 bits."""
    s = s.masked_fill(~visible, float("-inf"))
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (torch.log(total) + top).squeeze(-1)


def _prompt(st):
    """All sequences padded to the longest; grouped heads share their keys."""
    case, cu = st["case"], st["cu_seqlens"].long()
    h, hk, d, b, n = case["heads"], case["kv_heads"], case["dim"], case["seqs"], case["longest"]
    pos = torch.arange(n, device=cu.device)
    length = (cu[1:] - cu[:-1])[:, None]
    inside = pos[None] < length
    rows = torch.where(inside, cu[:-1, None] + pos, torch.zeros_like(pos))
    q = st["q"][rows].float().view(b, n, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    k = st["k"][rows].float().permute(0, 2, 3, 1)
    v = st["v"][rows].float().permute(0, 2, 1, 3)
    s = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(b, hk, h // hk, n, n)
    visible = inside[:, None, :]
    if case["causal"]:
        visible = visible & (pos[None, :] <= pos[:, None])
    o, lse = _softmax_v(s, v[:, :, None], visible[:, None, None])
    # Back to packed rows: packed token t is row t - cu[b] of its sequence b.
    t = st["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(b, device=cu.device), length[:, 0], output_size=t)
    at = torch.arange(t, device=cu.device) - cu[seq]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, h, d)[seq, at]
    lse = lse.permute(0, 3, 1, 2).reshape(b, n, h)[seq, at]
    return o.bfloat16(), lse


def _written(x, codes, scales, st):
    """The pool after the rows x [T, Hkv, d] went into their pages.  Quotients are formed in 64 bits: they lie on or
    next to the border between two codes."""
    case, page = st["case"], st["case"]["page"]
    cu, start = st["cu_seqlens"].long(), st["starts"].long()
    dev = cu.device
    j = start[:, None] // page + torch.arange(st["touched"], device=dev)  # [B, M] page numbers within the sequence
    end = start + cu[1:] - cu[:-1]
    valid = j * page < end[:, None]
    ids = torch.gather(st["table"].long(), 1, j.clamp(max=st["table"].shape[1] - 1))
    ids = torch.where(valid, ids, torch.full_like(ids, len(codes) - 1)).view(-1)
    pos = (j[:, :, None] * page + torch.arange(page, device=dev))  # [B, M, page]
    new = (pos >= start[:, None, None]) & (pos < end[:, None, None])
    rows = torch.where(new, cu[:-1, None, None] + pos - start[:, None, None], torch.zeros_like(pos)).view(-1, page)
    new = new.view(-1, 1, page, 1)
    value = torch.where(new, x[rows].permute(0, 2, 1, 3).float(), torch.zeros((), device=dev))  # [BM, Hkv, page, d]
    need = (value.abs().amax((2, 3)).double() / 127).float()
    begun = (j * page < start[:, None]) | ~valid
    old = scales[ids]
    scale = torch.where(begun.view(-1, 1), torch.maximum(old, need), need)
    wide = scale.double()[:, :, None, None]
    safe = torch.where(wide > 0, wide, torch.ones_like(wide))
    held = codes[ids]
    again = torch.round(held.double() * old.double()[:, :, None, None] / safe).clamp(-127, 127).to(torch.int8)
    again = torch.where((scale > old)[:, :, None, None] & begun.view(-1, 1, 1, 1)
                        & (pos.view(-1, 1, page, 1) < start.repeat_interleave(j.shape[1]).view(-1, 1, 1, 1)),
                        again, held)
    fresh = torch.round(value.double() / safe).clamp(-127, 127).to(torch.int8)
    codes[ids] = torch.where(new, fresh, again)
    scales[ids] = scale


def _write(st):
    _written(st["k"], st["k_cache"], st["k_scale"], st)
    _written(st["v"], st["v_cache"], st["v_scale"], st)
    page, cu = st["case"]["page"], st["read_cu"].long()
    dev, t = cu.device, st["read_total"]
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device=dev), cu[1:] - cu[:-1], output_size=t)
    pos = torch.arange(t, device=dev) - cu[seq] + st["read_starts"].long()[seq]
    ids = st["table"].long()[seq, pos // page]
    k = st["k_cache"][ids, :, pos % page].float() * st["k_scale"][ids][:, :, None]
    v = st["v_cache"][ids, :, pos % page].float() * st["v_scale"][ids][:, :, None]
    return k, v, st["k_scale"], st["v_scale"]


def _decode(st):
    """All histories padded to the table's width."""
    case, table = st["case"], st["table"].long().clamp(min=0)
    b, m, h, d = st["q"].shape
    hk, n = case["kv_heads"], table.shape[1] * case["page"]
    k = (st["k_cache"][table].float() * st["k_scale"][table][..., None, None]).permute(0, 2, 1, 3, 4).reshape(b, hk, n, d)
    v = (st["v_cache"][table].float() * st["v_scale"][table][..., None, None]).permute(0, 2, 1, 3, 4).reshape(b, hk, n, d)
    q = st["q"].float().view(b, m, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(b, hk, m, h // hk, n)
    last = st["seqlens"].long()[:, None] - m + torch.arange(m, device=table.device)  # [B, m]: the last key a token sees
    visible = torch.arange(n, device=table.device) <= last[..., None]
    o, lse = _softmax_v(s, v[:, :, None], visible[:, None, :, None])
    return o.permute(0, 2, 1, 3, 4).reshape(b, m, h, d).bfloat16(), lse.permute(0, 2, 1, 3).reshape(b, m, h)


# ----------------------------------------------------------------------- work
def work(case):
    h, hk, d = case.get("heads"), case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    t = sum(lengths)
    if case["kind"] == "prompt":
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lengths)
        return {"bytes": 2 * d * t * (2 * h + 2 * hk) + 4 * t * h + 4 * len(lengths), "flops": 4 * d * h * pairs}
    page = case["page"]
    if case["kind"] == "write":
        back = sum(a + n - a // page * page for a, n in zip(_held(case), lengths))
        # New rows in, their codes out; the touched rows' codes in again and their values out.
        return {"bytes": 2 * hk * d * (2 * t + t + back + 4 * back), "flops": 2 * hk * d * (3 * t + back)}
    pages = sum(-(-n // page) for n in lengths)
    m = case["new"]
    pairs = sum(max(0, n - m + 1 + i) for n in lengths for i in range(m))
    return {"bytes": 2 * hk * d * t + 8 * hk * pages + 4 * pages + len(lengths) * m * h * (4 * d + 4),
            "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------- exact
def _exact_rows(q, k, v, last):
    """One head: q [m, d] over k, v [n, d] in 64 bits; row i sees keys 0..last[i]."""
    n = k.shape[0]
    s = (q @ k.t()) / math.sqrt(q.shape[-1])
    s[torch.arange(n, device=q.device)[None] > last[:, None]] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.nan_to_num(torch.exp(s - lse[:, None]), nan=0.0)
    return p @ v, lse


def _exact_codes(x, s):
    return torch.clamp(torch.round(x / s), -127, 127) if s > 0 else torch.zeros_like(x)


def exact(case, seed):
    st = prepare(case, seed)
    lengths, hk, d = st["lengths"], case["kv_heads"], case["dim"]
    if case["kind"] == "prompt":
        group = case["heads"] // hk
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
        lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=DEVICE)
        at = 0
        for n in lengths:
            for i in range(case["heads"]):
                k, v = st["k"][at:at + n, i // group].double(), st["v"][at:at + n, i // group].double()
                for r in range(0, n, 4096):
                    e = min(n, r + 4096)
                    last = torch.arange(r, e, device=DEVICE) if case["causal"] else torch.full((e - r,), n, device=DEVICE)
                    o[at + r:at + e, i], lse[at + r:at + e, i] = _exact_rows(
                        st["q"][at + r:at + e, i].double(), k, v, last)
            at += n
        return o, lse
    page, table = case["page"], st["table"].tolist()
    if case["kind"] == "write":
        if sum(lengths) * hk // page > 20000 or case["seqs"] * hk > 4000:
            return None  # page by page it would take too long
        held, out = _held(case), []
        for x, codes, scales in ((st["k"], st["k_cache"], st["k_scale"]), (st["v"], st["v_cache"], st["v_scale"])):
            x, scales, parts, at = x.cpu().double(), scales.cpu().double(), [], 0
            for b, n in enumerate(lengths):
                first, end = held[b] // page, -(-(held[b] + n) // page)
                values = torch.zeros(((end - first) * page, hk, d), dtype=torch.float64)
                for j in range(first, end):
                    lo, hi = max(held[b], j * page), min(held[b] + n, (j + 1) * page)
                    block = x[at + lo - held[b]:at + hi - held[b]]
                    old = codes[table[b][j]].cpu().double()
                    for i in range(hk):
                        s = (block[:, i].abs().max() / 127).float().double()
                        here = values[(j - first) * page:(j + 1 - first) * page, i]
                        if lo > j * page:
                            s0 = scales[table[b][j], i].clone()
                            s = torch.maximum(s, s0)
                            here[:lo - j * page] = _exact_codes(old[i, :lo - j * page] * s0, s) * s
                        here[lo - j * page:hi - j * page] = _exact_codes(block[:, i], s) * s
                        scales[table[b][j], i] = s
                parts.append(values[:held[b] + n - first * page])
                at += n
            out.append((torch.cat(parts), scales))
        return out[0][0], out[1][0], out[0][1], out[1][1]
    b, m, h = st["q"].shape[:3]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros((b, m, h), dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(lengths):
        ids = st["table"][i, :-(-n // page)].long()
        last = torch.arange(n - m, n, device=DEVICE).repeat_interleave(h // hk)
        for c in range(hk):
            k = (st["k_cache"][ids, c].double() * st["k_scale"][ids, c].double()[:, None, None]).view(-1, d)[:n]
            v = (st["v_cache"][ids, c].double() * st["v_scale"][ids, c].double()[:, None, None]).view(-1, d)[:n]
            heads = slice(c * (h // hk), (c + 1) * (h // hk))
            rows, sums = _exact_rows(st["q"][i, :, heads].double().reshape(-1, d), k, v, last)
            o[i, :, heads], lse[i, :, heads] = rows.view(m, -1, d), sums.view(m, -1)
    return o, lse
