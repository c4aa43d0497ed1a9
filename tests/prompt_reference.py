"""Prompt attention in 64 bits, one sequence and query head at a time, with bounds on
the kernel's error; and the cache's planning on the host, from its definition."""
import math

import torch

D = PAGE = 128


def rows(T, H, seed, device="cuda", outliers=True):
    """bf16 [T, H, 128] ~ N(0, 1), four channels a head eight times as large."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g)
    if outliers:
        x = x * torch.where(torch.rand((1, H, D), generator=g) < 4 / D, 8.0, 1.0)
    return x.to(torch.bfloat16).to(device)


def starts(lens, device="cuda"):
    return torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=device)


def attention(Q, K, V, lens, causal=True, softcap=0.0, scale=None, prior=None):
    """O, lse in 64 bits and bounds on the error of each (rows behind the last sequence stay NaN).

    The score: the products are exact; 128 of them and the accumulator are added in fp32,
    each addition off by at most 2^-23 of what it holds (a tensor core may truncate):
    2^-16 of the sum of magnitudes.  The scale factor, its product and exp2: 2^-20 more
    of the probability.  A cap's tanh: 2^-20 of the capped score, which is at most
    the cap and at most the sum of magnitudes; below a cap of 64, 2^-20 of the cap
    (1 - 2 / (1 + 2^u): exp2 and reciprocal to 2^-22 each, two additions to 2^-24, halved at most).
    A probability is off by twice that (its own score and the largest one's) and by its
    rounding to bf16: 2^-8 relative.  n of them are added in fp32: 2^-23 n.  O rounds to
    bf16: 2^-8.  A prior enters with a weight that is off like a probability, unrounded."""
    T, Hq = Q.shape[:2]
    G = Hq // K.shape[1]
    scale = scale or 1.0 / math.sqrt(D)
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=Q.device)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=Q.device)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    lo = 0
    for n in lens:
        sl = slice(lo, lo + n)
        lo += n
        hide = torch.ones((n, n), dtype=torch.bool, device=Q.device).triu(1) if causal else None
        for h in range(Hq if n else 0):
            q, k, v = Q[sl, h].double(), K[sl, h // G].double(), V[sl, h // G].double()
            s, mag = q @ k.T * scale, q.abs() @ k.abs().T * scale
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            if causal:
                s, mag = s.masked_fill(hide, -math.inf), mag.masked_fill(hide, 0.0)
            top = mag.amax(-1)
            es = 2.0 ** -16 * top + 2.0 ** -20 * (1.0 + (torch.full_like(top, softcap) if softcap <= 64 else top.clamp(max=softcap)))
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            x, ax = p @ v, p @ v.abs()
            off = (2.0 ** -8 + 2 * es + 2.0 ** -23 * n)[:, None] * ax
            if prior is not None:
                b = prior[1][sl, h].double()
                po = torch.where(torch.isinf(b)[:, None], 0.0, prior[0][sl, h].double())
                both = torch.logaddexp(z, b)
                wz, wb = torch.exp(z - both), torch.exp(b - both)
                eb = es + 2.0 ** -22 * torch.where(torch.isinf(b), 0.0, b.abs())
                x = wz[:, None] * x + wb[:, None] * po
                off = wz[:, None] * off + (2 * eb)[:, None] * (wz[:, None] * ax + wb[:, None] * po.abs())
                es, z = eb, both
            o[sl, h], lse[sl, h] = x, z
            eo[sl, h] = off + 2.0 ** -8 * x.abs() + 2.0 ** -126
            el[sl, h] = es + 2.0 ** -22 * z.abs() + 2.0 ** -20 + 2.0 ** -23 * n
    return o, lse, eo, el


def within(got, ref, bound, what):
    """Everywhere at most `bound` off; what is not finite is the same."""
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin) and torch.equal(torch.isnan(got), torch.isnan(ref)), what
    over = ((got - ref).abs() - bound)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: off by {float(over.max()):.3e} more than allowed"


def up(n):
    return -(-n // PAGE)


def free_pages(table, held, pages):
    named = {p for row, m in zip(table, held) for p in row[:up(m)]}
    return [p for p in range(pages) if p not in named]


def plan(table, held, news, pages, T):
    """(table, length, start, slot, position, status) of lists; a plan that cannot be made whole leaves all but start as it is."""
    B, cols = len(table), len(table[0])
    bad = any(m < 0 or n < 0 or m + n > cols * PAGE for m, n in zip(held, news)) or sum(news) > T
    if bad:
        return table, None, [0] * (B + 1), [], [], 1
    free = free_pages(table, held, pages)
    if sum(up(m + n) - up(m) for m, n in zip(held, news)) > len(free):
        return table, None, [0] * (B + 1), [], [], 6
    free, table = iter(free), [row[:] for row in table]
    start, slot, position = [0], [], []
    for row, m, n in zip(table, held, news):
        for j in range(up(m), up(m + n)):
            row[j] = next(free)
        start.append(start[-1] + n)
        position += range(m, m + n)
        slot += [row[i // PAGE] * PAGE + i % PAGE if 0 <= row[i // PAGE] < pages else -1 for i in range(m, m + n)]
    return table, [m + n for m, n in zip(held, news)], start, slot, position, 0


def fresh(table, held, pages, budget, dst):
    free = iter(free_pages(table, held, pages))
    return [[next(free) if j < up(min(m, budget)) else x for j, x in enumerate(row)] for m, row in zip(held, dst)]
