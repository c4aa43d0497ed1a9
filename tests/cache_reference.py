"""The 8-bit cache's operators in 64 bits on the CPU, sequence by sequence and
head by head, from their definition; seeded cases; and the error bounds that the
kernels' arithmetic allows."""
import math
from dataclasses import dataclass

import torch

D = PAGE = 128
SMIN = 2.0 ** -120


def decode(codes):
    return codes.view(torch.float8_e4m3fn).double()


def encode(x):
    """E4M3 codes of float64 values that fp32 holds exactly and |x| <= 448; NaN for what is not finite."""
    x = torch.where(torch.isfinite(x), x, math.nan)
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8)


def scale_for(amax):
    s = SMIN
    while 448.0 * s < amax:
        s *= 2.0
    return s


@dataclass
class Case:
    """A cache on the CPU with its batch; `on` moves it to a device as the binding's Cache."""
    k8: torch.Tensor
    v8: torch.Tensor
    sk: torch.Tensor
    sv: torch.Tensor
    table: torch.Tensor
    length: torch.Tensor
    start: torch.Tensor

    def clone(self):
        return Case(*(getattr(self, f).clone() for f in self.__dataclass_fields__))

    def on(self, V, device="cuda"):
        t = [getattr(self, f).to(device) for f in ("k8", "v8", "sk", "sv", "table", "length")]
        return V.Cache(*t), self.start.to(device)


def random_codes(g, shape):
    return (torch.randn(shape, generator=g) * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def make_case(lens, news, H, cols=None, seed=0, spare=1, scales=(-6, -7)):
    """Sequences of the given lengths over shuffled pages of random codes; slots
    behind a sequence's last token and spare pages hold NaN codes."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-m // PAGE) for m in lens]
    pages = sum(need) + spare
    cols = cols or max(max(need), 1)
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    k8 = torch.full((pages, H, PAGE, D), 0x7F, dtype=torch.uint8)
    v8 = k8.clone()
    at = 0
    for b, (m, c) in enumerate(zip(lens, need)):
        for j in range(c):
            p = int(order[at])
            at += 1
            table[b, j] = p
            r = min(PAGE, m - j * PAGE)
            k8[p, :, :r] = random_codes(g, (H, r, D))
            v8[p, :, :r] = random_codes(g, (H, r, D))
    pick = torch.tensor([2.0 ** e for e in scales])
    sk = pick[torch.randint(len(scales), (pages, H), generator=g)]
    sv = pick[torch.randint(len(scales), (pages, H), generator=g)]
    start = torch.tensor([sum(news[:b]) for b in range(len(lens) + 1)], dtype=torch.int32)
    return Case(k8, v8, sk, sv, table, torch.tensor(lens, dtype=torch.int32), start)


def rows(T, H, seed, strided=False, outliers=True, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H + 2 if strided else H, D), generator=g)
    if outliers:
        x = x * torch.where(torch.rand((1, x.shape[1], D), generator=g) < 4 / D, 8.0, 1.0)
    x = x.to(torch.bfloat16).to(device)
    return x[:, 1:H + 1] if strided else x


def seq_values(c, b, h, codes, scale):
    m = int(c.length[b])
    if m == 0:
        return torch.zeros((0, D), dtype=torch.float64)
    p = c.table[b, :-(-m // PAGE)].long()
    return (decode(codes[p, h]) * scale[p, h].double()[:, None, None]).reshape(-1, D)[:m]


def seq_scores(c, Q, b, h, G, causal, softcap, scale):
    """Scores [n, G, len] (-inf where not visible) and the sum of the products' magnitudes, largest over the visible keys."""
    lo, hi, m = int(c.start[b]), int(c.start[b + 1]), int(c.length[b])
    k = seq_values(c, b, h, c.k8, c.sk)
    q = Q[lo:hi, h * G:(h + 1) * G].double()
    s = torch.einsum("igd,kd->igk", q, k) * scale
    mag = torch.einsum("igd,kd->igk", q.abs(), k.abs()) * scale
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    if causal:
        hide = torch.arange(m) > (torch.arange(hi - lo) + m - (hi - lo))[:, None]
        s = s.masked_fill(hide[:, None], -math.inf)
        mag = mag.masked_fill(hide[:, None], 0.0)
    return s, mag


def attention(c, Q, causal=True, softcap=0.0, scale=None):
    """O, lse in 64 bits and bounds on the error of each.

    The score: products are exact, 128 of them and the accumulator are added in
    fp32, each addition off by at most 2^-23 of what it holds (a tensor core may
    truncate): 2^-16 of the sum of magnitudes; the scale factors' and exp2's
    roundings 2^-20 more of the probability, a cap's tanh 2^-20 of the capped score,
    which is at most the cap and at most the sum of magnitudes.  A probability is off by twice that (its own score and the
    largest one's) and by its rounding to fp16: 2^-11, or 2^-25 absolute.  O
    rounds to bf16: 2^-8."""
    T, Hq = Q.shape[:2]
    H = c.k8.shape[1]
    G = Hq // H
    scale = scale or 1.0 / math.sqrt(D)
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(len(c.length)):
        lo, hi = int(c.start[b]), int(c.start[b + 1])
        for h in range(H):
            s, mag = seq_scores(c, Q, b, h, G, causal, softcap, scale)
            v = seq_values(c, b, h, c.v8, c.sv)
            if s.shape[-1] == 0:
                z = torch.full(s.shape[:2], -math.inf, dtype=torch.float64)
                p = s
                top = torch.zeros(s.shape[:2], dtype=torch.float64)
            else:
                z = torch.logsumexp(s, -1)
                p = torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[..., None])
                top = mag.amax(-1)
            es = 2.0 ** -16 * top + 2.0 ** -20 * (1.0 + top.clamp(max=softcap))
            sl = slice(h * G, (h + 1) * G)
            o[lo:hi, sl] = p @ v
            lse[lo:hi, sl] = z
            el[lo:hi, sl] = es + 2.0 ** -22 * torch.where(torch.isinf(z), 0.0, z.abs()) + 2.0 ** -20
            # below 2^-14 of the largest a probability rounds by up to 2^-25 of the largest, and never by more than itself
            small = torch.minimum(p, 2.0 ** -25 * p.amax(-1, keepdim=True)) if len(v) else p
            eo[lo:hi, sl] = (2.0 ** -8 * o[lo:hi, sl].abs() + (2.0 ** -11 + 2 * es)[..., None] * (p @ v.abs()) + small @ v.abs())
    return o, lse, eo, el


def weigh(c, Q, lse, weight, causal=True, softcap=0.0, scale=None):
    """The weights in 64 bits and bounds: each exp(s - lse) as above without the
    rounding to fp16, the subtraction rounding to 2^-24 of its terms; sums of R
    terms in fp32."""
    H = c.k8.shape[1]
    G = Q.shape[1] // H
    scale = scale or 1.0 / math.sqrt(D)
    w, e = weight.double(), torch.zeros(weight.shape, dtype=torch.float64)
    for b in range(len(c.length)):
        lo, hi, m = int(c.start[b]), int(c.start[b + 1]), int(c.length[b])
        if m == 0 or hi == lo:
            continue
        p = c.table[b, :-(-m // PAGE)].long()
        for h in range(H):
            s, mag = seq_scores(c, Q, b, h, G, causal, softcap, scale)
            z = lse[lo:hi, h * G:(h + 1) * G].double()[..., None]
            x = torch.where(s > -math.inf, torch.exp(s - z), 0.0)
            off = 2.0 ** -16 * mag + 2.0 ** -20 * (1.0 + mag.clamp(max=softcap)) + 2.0 ** -22 * (s.abs().nan_to_num(0, 0, 0) + z.abs().nan_to_num(0, 0, 0))
            for t, y in ((w, x.sum((0, 1))), (e, (x * off).sum((0, 1)) + 2.0 ** -22 * x.sum((0, 1)))):
                flat = t[p, h].reshape(-1)
                flat[:m] += y
                t[p, h] = flat.view(-1, PAGE)
    return w, e + 2.0 ** -23 * w.abs()


def append(c, K, V):
    """In place: codes and scales after the rows K, V arrive."""
    for X, codes, scale in ((K, c.k8, c.sk), (V, c.v8, c.sv)):
        for b in range(len(c.length)):
            lo, hi, m = int(c.start[b]), int(c.start[b + 1]), int(c.length[b])
            first = m - (hi - lo)
            for t in range(first // PAGE, -(-m // PAGE) if hi > lo else 0):
                a, z = max(first, t * PAGE), min(m, (t + 1) * PAGE)
                p, r = int(c.table[b, t]), a - t * PAGE
                for h in range(codes.shape[1]):
                    x = X[lo + a - first:lo + z - first, h].double()
                    fin = x[torch.isfinite(x)]
                    s = scale_for(float(fin.abs().max()) if fin.numel() else 0.0)
                    if r > 0 and float(scale[p, h]) > s:
                        s = float(scale[p, h])
                    if r > 0:
                        codes[p, h, :r] = encode(decode(codes[p, h, :r]) * (float(scale[p, h]) / s))
                    codes[p, h, r:r + z - a] = encode(x / s)
                    scale[p, h] = s


def evict(c, weight, dst, budget, recent, kept):
    """In place (codes, scales, weight, kept); returns the new lengths."""
    old = c.clone()
    w_old = weight.clone()
    new_len = torch.clamp(c.length, max=budget)
    for b in range(len(c.length)):
        m, stay = int(c.length[b]), int(new_len[b])
        r = min(m, recent)
        for h in range(c.k8.shape[1]):
            p = c.table[b, :-(-m // PAGE)].long()
            wt = w_old[p, h].reshape(-1)[:m]
            key = torch.where(torch.isnan(wt), -math.inf, wt)[:m - r].tolist()
            heavy = sorted(range(m - r), key=lambda t: (-key[t], t))[:stay - r]
            at = sorted(heavy) + list(range(m - r, m))
            kept[b, h, :stay] = torch.tensor(at, dtype=torch.int32)
            for j in range(0, stay, PAGE):
                sel = torch.tensor(at[j:j + PAGE])
                d = int(dst[b, j // PAGE])
                for codes, scale, oc, os in ((c.k8, c.sk, old.k8, old.sk), (c.v8, c.sv, old.v8, old.sv)):
                    x = seq_values(old, b, h, oc, os)[sel]
                    fin = x[torch.isfinite(x)]
                    s = scale_for(float(fin.abs().max()) if fin.numel() else 0.0)
                    codes[d, h, :len(sel)] = encode(x / s)
                    scale[d, h] = s
                weight[d, h, :len(sel)] = wt[sel]
    return new_len
