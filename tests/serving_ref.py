"""Plain 64-bit forms of the serving operators, for the tests (CPU tensors)."""
import torch


def attention(q, k, v, scale, last):
    """One head: q [m,d] over k, v [n,d]; row i sees keys 0..last[i].  Returns O, LSE, and per
    row A = sum_j p_j |v_j| and the largest scale * sum_e |q_e k_e| of a visible key, which the
    rounding bounds are built from."""
    q, k, v = q.double(), k.double(), v.double()
    n = k.shape[0]
    seen = torch.arange(n)[None] <= torch.as_tensor(last)[:, None]
    s = torch.where(seen, scale * (q @ k.t()), -torch.inf)
    lse = torch.logsumexp(s, -1) if n else torch.full((q.shape[0],), -torch.inf, dtype=torch.float64)
    p = torch.where(seen, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]), 0.0)
    size = torch.where(seen, scale * (q.abs() @ k.abs().t()), 0.0)
    size = size.amax(-1) if n else torch.zeros(q.shape[0], dtype=torch.float64)
    return p @ v, lse, p @ v.abs(), size


def score_error(size, d):
    """|s - exact s| of a product over d terms summed in 32 bits in any order: every one of the
    at most d + 1 additions and the scale's two multiplications round by 2^-24 of a value no larger
    than the sum of magnitudes; twice that for a tensor core that truncates."""
    return (d + 4) * 2.0 ** -23 * size


def output_bound(o, a, size, d, p_unit):
    """|O - exact O| where P is rounded to p_unit relative, O to BF16 (2^-8), every score is off by
    score_error (which moves each p_j / sum p by at most twice that), and 2^-18 covers the FP32
    sums, exponentials (2^-22 each) and the division."""
    e = score_error(size, d)[:, None]
    return (p_unit + 2 * e + 2.0 ** -18) * a + 2.0 ** -8 * (o.abs() + (p_unit + 2 * e) * a) + 1e-30


def lse_bound(lse, size, d):
    """The scores' error, a sum and a logarithm in 32 bits."""
    return score_error(size, d) + 2.0 ** -20 * (1 + lse.abs())


def rint_quotient(x, s):
    """rint(x / s) clamped to +-127 of doubles x, s > 0 (x / s is near enough to exact: operands
    of at most 31 bits, so a quotient next to a border is off by far more than 2^-53)."""
    return torch.clamp(torch.round(x / s), -127, 127)


def append(rows, codes, scales, table, start):
    """Write rows [n, Hkv, d] behind position `start` of a sequence with pages `table`, in place:
    codes [P, Hkv, page, d] int8, scales [P, Hkv] float32."""
    n, hk, _ = rows.shape
    page = codes.shape[2]
    x = rows.double()
    for j in range(start // page, -(-(start + n) // page) if n else 0):
        lo, hi = max(start, j * page), min(start + n, (j + 1) * page)
        if lo >= hi:
            continue
        p = table[j]
        for h in range(hk):
            block = x[lo - start:hi - start, h]
            finite = torch.where(block.isfinite(), block, 0.0)
            s = (finite.abs().max() / 127).float()
            if lo > j * page:
                s0 = scales[p, h].clone()
                s = torch.maximum(s, s0)
                if s > s0:
                    old = codes[p, h, :lo - j * page].double() * s0.double()
                    codes[p, h, :lo - j * page] = rint_quotient(old, s.double()).to(torch.int8)
            if s > 0:
                c = rint_quotient(torch.where(block.isnan(), 0.0, block), s.double())
            else:
                c = torch.zeros_like(block)
            codes[p, h, lo - j * page:hi - j * page] = c.to(torch.int8)
            scales[p, h] = s


def cached(codes, scales, table, n):
    """Values [n, Hkv, d] (float64) of the first n positions of a sequence."""
    page, hk, d = codes.shape[2], codes.shape[1], codes.shape[3]
    ids = list(table[:-(-n // page)])
    v = codes[ids].double() * scales[ids].double()[:, :, None, None]
    return v.permute(0, 2, 1, 3).reshape(-1, hk, d)[:n]


def reserve(table, held, wanted, stack, free, page, T, pages):
    """A step of attn_cache_reserve on lists, one request after the other: table [B][max_blocks] and stack
    [pages] are updated; returns (lens, cu, slots, positions, free)."""
    up = lambda n: -(-n // page)  # noqa: E731
    room = len(table[0]) * page
    wanted = [w if 0 <= h <= room and 0 <= w <= room else h for h, w in zip(held, wanted)]
    fine = [0 <= h <= room for h in held]
    valid = lambda p: p if 0 <= p < pages else -1  # noqa: E731
    free = min(max(free, 0), pages)
    for b, (h, w) in enumerate(zip(held, wanted)):
        for j in range(up(w), up(h)) if fine[b] else ():
            if free < pages:
                stack[free] = valid(table[b][j])
            table[b][j] = -1
            free += 1
    free = min(free, pages)
    lens, asked, took = [], 0, 0
    for b, (h, w) in enumerate(zip(held, wanted)):
        need = max(0, up(w) - up(h)) if fine[b] else 0
        asked += need
        serve = need == 0 or asked <= free
        took += need * serve
        lens.append(w if serve else h)
    free -= took
    at, cu, slots, positions = free, [0], [], []
    for b, (h, w) in enumerate(zip(held, wanted)):
        serve = lens[b] == w
        for j in range(up(h), up(w)) if fine[b] else ():
            table[b][j] = valid(stack[at]) if serve else -1
            at += serve
        for t in range(h, w):
            p = valid(table[b][t // page])
            slots.append(p * page + t % page if serve and p >= 0 else -1)
            positions.append(t)
        cu.append(len(slots))
    fill = [-1] * max(0, T - len(slots))
    return lens, cu, (slots + fill)[:T], (positions + fill)[:T], free
