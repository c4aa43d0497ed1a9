"""The 8-bit cache operators as measured workloads: append, attention, weigh and evict.

The cache: k8, v8 E4M3 bytes [pages][H][128][128]; sk, sv fp32 powers of two
[pages][H]; table int32 [B][cols] (page of tokens 128 j .. 128 j + 127 of
sequence b, -1 where there is none); length int32 [B], the tokens held with the
new ones included.  The rows start[b] .. start[b+1]-1 of K, V and Q belong to
sequence b; row i of its n sits at slot length - n + i.

`run` computes an operator in elementary torch operations where `own` is false
and by the library's entry points where it is true; `exact` computes it in 64
bits, sequence by sequence, from the definition.
"""
import math

import torch

own = False

D = 128
PAGE = 128
SMIN = 2.0 ** -120      # smallest page scale
EMAX = 448.0            # largest E4M3 value


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(name, op, B, Hq, Hkv, n, length, ragged=False, causal=False, softcap=0.0, strided=False, budget=0, recent=0):
    c = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "n": n, "length": length, "ragged": ragged, "causal": causal,
         "softcap": softcap, "strided": strided, "budget": budget, "recent": recent}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one new token for each of a few short sequences: launch latency
        _case("append_token", "append", 16, 8, 8, 1, 1000, ragged=True),
        # a quarter of the 70,656-token video arrives as one chunk, K and V as views of a fused projection
        _case("append_chunk", "append", 1, 40, 40, 17664, 40001, strided=True),
        # one token, one short sequence, own KV head for every query head: latency
        _case("attend_token_short", "attention", 1, 24, 24, 1, 300, causal=True),
        # a batch of sequences at different lengths, five query heads to a KV head: the ordinary decode step
        _case("attend_token_batch", "attention", 32, 40, 8, 1, 32768, ragged=True, causal=True),
        # one very long sequence, 40 heads: a gigabyte of cache for one token
        _case("attend_token_long", "attention", 1, 40, 40, 1, 131072, causal=True),
        # a few tokens a sequence checked at once, capped scores
        _case("attend_few_capped", "attention", 8, 40, 8, 5, 16383, ragged=True, causal=True, softcap=30.0, strided=True),
        # a sixteenth of the 70,656-token video attends to all of it, both ways
        _case("attend_frames", "attention", 1, 8, 8, 4416, 70656),
        # prompts of different lengths behind short prefixes, causal, shared KV heads
        _case("attend_prompts", "attention", 4, 32, 8, 2900, 4097, ragged=True, causal=True),
        # the decode step's weights for eviction
        _case("weigh_token_batch", "weigh", 32, 40, 8, 1, 32768, ragged=True, causal=True),
        # a chunk's weights over the whole video
        _case("weigh_frames", "weigh", 1, 8, 8, 1104, 70656),
        # a short history cut to a few hundred tokens in every head
        _case("evict_short", "evict", 2, 24, 24, 1, 1000, ragged=True, budget=300, recent=37),
        # long prompts cut to an eighth
        _case("evict_prompts", "evict", 4, 40, 8, 1, 32768, ragged=True, budget=4096, recent=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "weigh", "evict"])
    heads = rng.choice([(8, 8), (24, 24), (40, 40), (40, 8), (32, 8), (16, 1), (12, 4), (7, 1)])
    Hq, Hkv = heads
    causal = rng.random() < 0.7
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    strided = rng.random() < 0.5
    if op == "append":
        n = _log_int(rng, 1, 8000)
        B = _log_int(rng, 1, max(1, min(64, 16000 // n)))
        length = n + _log_int(rng, 1, 8000) - 1
        return _case("", op, B, Hkv, Hkv, n, length, ragged=rng.random() < 0.7, strided=strided)
    if op == "evict":
        length = _log_int(rng, 2, 40000)
        B = _log_int(rng, 1, max(1, min(16, 100000 // length)))
        budget = _log_int(rng, 1, max(1, length // 2))
        recent = rng.randint(0, budget)
        return _case("", op, B, Hkv, Hkv, 1, length, ragged=True, budget=budget, recent=recent)
    if rng.random() < 0.55:   # single tokens
        n = 1
        length = _log_int(rng, 1, 100000)
        B = _log_int(rng, 1, max(1, min(64, 5000000 // (length * Hkv))))
    else:
        n = _log_int(rng, 2, 1000 if op == "weigh" else 2900)
        length = n + _log_int(rng, 1, 16000)
        B = _log_int(rng, 1, max(1, min(16, 2000000000 // (n * length * Hq))))
    return _case("", op, B, Hq, Hkv, n, length, ragged=rng.random() < 0.7, causal=causal, softcap=cap, strided=strided)


def _lens(case):
    """New rows and tokens held of each sequence: spread evenly from a tenth of the largest to all of it where ragged."""
    news, lens = [], []
    for b in range(case["B"]):
        f = 1.0 - 0.9 * ((b * 0.6180339887498949) % 1.0) if case["ragged"] else 1.0
        g = 1.0 - 0.9 * ((b * 0.4142135623730951) % 1.0) if case["ragged"] else 1.0
        n = max(1, int(case["n"] * g))
        news.append(n)
        lens.append(max(n, int(case["length"] * f)))
    return news, lens


def _visible(case):
    """Query-key pairs of one query head."""
    news, lens = _lens(case)
    if not case["causal"]:
        return sum(n * m for n, m in zip(news, lens))
    return sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(news, lens))


def work(case):
    news, lens = _lens(case)
    T, L, Hq, Hkv, B = sum(news), sum(lens), case["Hq"], case["Hkv"], case["B"]
    index = 4 * (2 * B + 1) + 4 * sum(-(-m // PAGE) for m in lens)
    pages = sum(-(-m // PAGE) for m in lens)
    if case["op"] == "append":
        return {"bytes": T * Hkv * D * (4 + 2) + index, "flops": 4 * T * Hkv * D}
    if case["op"] == "attention":
        return {"bytes": 2 * L * Hkv * D + 8 * pages * Hkv + T * Hq * (4 * D + 4) + index, "flops": 4 * D * Hq * _visible(case)}
    if case["op"] == "weigh":
        return {"bytes": L * Hkv * (D + 8) + 4 * pages * Hkv + T * Hq * (2 * D + 4) + index, "flops": 2 * D * Hq * _visible(case)}
    kept = sum(min(m, case["budget"]) for m in lens)
    return {"bytes": 4 * L * Hkv + kept * Hkv * (4 * D + 8) + index, "flops": 4 * kept * Hkv * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _rows(g, T, H, strided, outliers):
    """bf16 [T][H][128] ~ N(0, 1), four channels a head eight times as large where `outliers`; a view into wider rows where strided."""
    x = torch.randn((T, H + 2 if strided else H, D), generator=g, device="cuda")
    if outliers:
        x = x * torch.where(torch.rand((1, x.shape[1], D), generator=g, device="cuda") < 4 / D, 8.0, 1.0)
    x = x.to(torch.bfloat16)
    return x[:, 1:H + 1] if strided else x


def _codes(g, pages, H, std):
    """E4M3 codes of N(0, std^2), page by page so that little is held at once."""
    out = torch.empty((pages, H, PAGE, D), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (H * PAGE * D))
    for p in range(0, pages, step):
        x = torch.randn((min(step, pages - p), H, PAGE, D), generator=g, device="cuda")
        out[p:p + step] = (x * std).clamp(-EMAX, EMAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    news, lens = _lens(case)
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    need = [-(-m // PAGE) for m in lens]
    fresh = [-(-min(m, case["budget"]) // PAGE) for m in lens]
    pages = sum(need) + sum(fresh) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)

    def table(counts, at):
        rows = []
        for c in counts:
            rows.append(torch.nn.functional.pad(order[at:at + c], (0, max(counts) - c), value=-1))
            at += c
        return torch.stack(rows).contiguous(), at

    # codes of unit-variance rows whose page scale is 2^-6 or 2^-7
    st = {"case": dict(case), "k8": _codes(g, pages, Hkv, 64.0), "v8": _codes(g, pages, Hkv, 64.0)}
    for s in ("sk", "sv"):
        st[s] = torch.where(torch.rand((pages, Hkv), generator=g, device="cuda") < 0.5, 2.0 ** -6, 2.0 ** -7)
    st["table"], at = table(need, 0)
    st["length"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["start"] = torch.tensor([sum(news[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    T = sum(news)
    op = case["op"]
    if op == "append":
        st["K"] = _rows(g, T, Hkv, case["strided"], True)
        st["V"] = _rows(g, T, Hkv, case["strided"], False)
        return st
    # what follows a sequence's last token in its last page may hold anything
    for b in range(B):
        if lens[b] % PAGE:
            p = int(st["table"][b, need[b] - 1])
            st["k8"][p, :, lens[b] % PAGE:] = 0x7F
            st["v8"][p, :, lens[b] % PAGE:] = 0x7F
    if op == "evict":
        st["weight"] = torch.empty((pages, Hkv, PAGE), device="cuda").exponential_(1.0, generator=g)
        # a part of the tokens never got any weight: ties
        st["weight"][torch.rand(st["weight"].shape, generator=g, device="cuda") < 0.2] = 0.0
        st["fresh"], _ = table(fresh, at)
        st["kept"] = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device="cuda")
        return st
    st["Q"] = _rows(g, T, Hq, case["strided"], True)
    st["ws"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")   # scratch that a server keeps
    if op == "weigh":
        st["lse"] = _softmax(st, False)[1]
        st["weight"] = torch.empty((pages, Hkv, PAGE), device="cuda").exponential_(1.0, generator=g)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _encode(x, s):
    """E4M3 codes of x / s (exact: s is a power of two); NaN where x is not finite."""
    y = torch.where(torch.isfinite(x), x / s, math.nan)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _scale_of(amax):
    """The smallest power of two that holds amax within 448, at least 2^-120."""
    m, e = torch.frexp(amax.double() / EMAX)
    s = torch.ldexp(torch.ones_like(m), e - (m == 0.5).int()).clamp_min(SMIN)
    return torch.where(amax > 0, s, SMIN).float()


def _tiles(st, codes, scale):
    """Values of every sequence's tokens, fp32 [B][H][cols * 128][128], 0 behind its last token."""
    t = st["table"].long().clamp_min(0)
    x = _decode(codes[t]) * scale[t][..., None, None]
    B, C, H = x.shape[:3]
    x = x.permute(0, 2, 1, 3, 4).reshape(B, H, C * PAGE, D)
    slot = torch.arange(C * PAGE, device=x.device)
    return torch.where((slot < st["length"][:, None])[:, None, :, None], x, 0.0)


def _scores(st):
    """Scores fp32 [B][Hkv][n G][cols * 128], -inf where a key is not visible, and the new rows' places."""
    c = st["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    G, nmax, T = Hq // Hkv, c["n"], st["Q"].shape[0]
    start, length = st["start"].long(), st["length"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(nmax, device="cuda")
    q = st["Q"][(start[:-1, None] + i).clamp_max(T - 1)].float()                  # [B][nmax][Hq][D]
    B = q.shape[0]
    q = q.view(B, nmax, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nmax * G, D)
    k = _tiles(st, st["k8"], st["sk"])
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    if c["softcap"] > 0:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    slot = torch.arange(k.shape[2], device="cuda")
    last = (length - n)[:, None] + i if c["causal"] else (length - 1)[:, None].expand(B, nmax)
    last = torch.where(i < n[:, None], torch.minimum(last, length[:, None] - 1), -1)
    seen = slot <= last[..., None]                                                # [B][nmax][slots]
    seen = seen[:, None, :, None].expand(B, Hkv, nmax, G, slot.numel()).reshape(s.shape)
    s = torch.where(seen, s, -math.inf)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return s, b, t - start[b]


def _unpad(x, st, b, i):
    """[B][Hkv][nmax G][...] -> [T][Hq][...]"""
    c = st["case"]
    B, Hkv, rows = x.shape[:3]
    x = x.reshape(B, Hkv, c["n"], rows // c["n"], *x.shape[3:]).transpose(1, 2)
    return x[b, i].reshape(b.numel(), c["Hq"], *x.shape[4:]).contiguous()


def _softmax(st, values):
    s, b, i = _scores(st)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = torch.exp(s - m)
    del s
    l = p.sum(-1, keepdim=True)
    lse = _unpad((torch.log(l) + m).squeeze(-1), st, b, i)
    if not values:
        return None, lse
    o = (p @ _tiles(st, st["v8"], st["sv"])) / torch.where(l > 0, l, 1.0)
    return _unpad(o, st, b, i).to(torch.bfloat16), lse


def _append_side(st, codes, scale, X):
    start, length, table = st["start"].long(), st["length"].long(), st["table"].long()
    n = start[1:] - start[:-1]
    first = length - n                                             # the first new slot
    cols = -(-st["case"]["n"] // PAGE) + 1                         # pages that new rows may reach
    col = (first // PAGE)[:, None] + torch.arange(cols, device="cuda")
    slot = col[..., None] * PAGE + torch.arange(PAGE, device="cuda")                  # [B][cols][128]
    new = (slot >= first[:, None, None]) & (slot < length[:, None, None])
    row = (start[:-1, None, None] + slot - first[:, None, None]).clamp(0, X.shape[0] - 1)
    x = torch.where(new[..., None, None], X[row].float(), 0.0).transpose(2, 3)        # [B][cols][H][128][D]
    page = table.gather(1, col.clamp_max(table.shape[1] - 1)).clamp_min(0)
    old = slot < first[:, None, None]
    had = old.any(-1)[..., None]                                                      # [B][cols][1]
    before = codes[page]
    amax = torch.where(torch.isfinite(x), x, 0.0).abs().amax((-1, -2))
    s_old = scale[page]
    s = torch.where(had, torch.maximum(_scale_of(amax), s_old), _scale_of(amax))
    kept = _encode(_decode(before) * s_old[..., None, None], s[..., None, None])
    code = torch.where(new[:, :, None, :, None], _encode(x, s[..., None, None]),
                       torch.where(old[:, :, None, :, None], kept, before))
    touched = new.any(-1)
    codes[page[touched]] = code[touched]
    scale[page[touched]] = s[touched]


def _append(st):
    _append_side(st, st["k8"], st["sk"], st["K"])
    _append_side(st, st["v8"], st["sv"], st["V"])


def _weigh(st):
    s, b, i = _scores(st)
    c = st["case"]
    B, Hkv, rows, slots = s.shape
    G = c["Hq"] // Hkv
    start = st["start"].long()
    t = (start[:-1, None] + torch.arange(c["n"], device="cuda")).clamp_max(st["lse"].shape[0] - 1)
    lse = st["lse"][t].view(B, c["n"], Hkv, G).transpose(1, 2).reshape(B, Hkv, rows, 1)
    p = torch.where(s > -math.inf, torch.exp(s - lse), 0.0).sum(2)                # [B][Hkv][slots]
    p = p.view(B, Hkv, slots // PAGE, PAGE).transpose(1, 2)                       # [B][cols][Hkv][128]
    live = st["table"] >= 0
    page = st["table"].long()[live]
    st["weight"][page] = st["weight"][page] + p[live]


def _move(codes, scale, page, head, at, there, fresh, live):
    """The tokens at (page, head, at) go to the pages `fresh`, with scales of their own."""
    B, F, H = there.shape[:3]
    x = (_decode(codes[page, head, at]) * scale[page, head][..., None]).view(B, H, F, PAGE, D).transpose(1, 2)
    s = _scale_of(torch.where(there[..., None] & torch.isfinite(x), x, 0.0).abs().amax((-1, -2)))
    code = torch.where(there[..., None], _encode(x, s[..., None, None]), codes[fresh.clamp_min(0)])
    codes[fresh[live]] = code[live]
    scale[fresh[live]] = s[live]


def _evict(st):
    c = st["case"]
    table, fresh, length = st["table"].long().clamp_min(0), st["fresh"].long(), st["length"].long()
    B, C = table.shape
    H, budget, F = c["Hkv"], c["budget"], fresh.shape[1]
    stays = torch.clamp(length, max=budget)                                       # tokens kept
    recent = torch.clamp(length, max=c["recent"])
    w = st["weight"][table].transpose(1, 2).reshape(B, H, C * PAGE)
    slot = torch.arange(C * PAGE, device="cuda")
    older = slot < (length - recent)[:, None]
    key = torch.where(older[:, None] & ~torch.isnan(w), w, -math.inf)
    rank = torch.sort(key, dim=-1, descending=True, stable=True).indices          # heaviest first, ties to the lowest slot
    place = torch.empty_like(rank).scatter_(-1, rank, slot.expand_as(rank).contiguous())
    keep = older[:, None] & (place < (stays - recent)[:, None, None])
    keep |= (~older & (slot < length[:, None]))[:, None]
    at = torch.sort(torch.where(keep, slot, C * PAGE), dim=-1).values             # kept slots in order, then the rest
    at = torch.nn.functional.pad(at, (0, F * PAGE), value=C * PAGE)[..., :F * PAGE]
    real = at < C * PAGE
    at = torch.where(real, at, 0)
    page = table.gather(1, (at // PAGE).reshape(B, -1)).view(at.shape)
    head = torch.arange(H, device="cuda")[:, None]
    live = fresh >= 0
    there = real.view(B, H, F, PAGE).transpose(1, 2)
    _move(st["k8"], st["sk"], page, head, at % PAGE, there, fresh, live)
    _move(st["v8"], st["sv"], page, head, at % PAGE, there, fresh, live)
    wn = st["weight"][page, head, at % PAGE].view(B, H, F, PAGE).transpose(1, 2)
    st["weight"][fresh[live]] = torch.where(there, wn, st["weight"][fresh.clamp_min(0)])[live]
    count = torch.arange(budget, device="cuda") < stays[:, None]
    st["kept"].copy_(torch.where(count[:, None], torch.nn.functional.pad(at, (0, budget))[..., :budget], st["kept"]))
    return stays.to(torch.int32)


def _plain(st):
    op = st["case"]["op"]
    if op == "append":
        _append(st)
        return None
    if op == "attention":
        return _softmax(st, True)
    if op == "weigh":
        _weigh(st)
        return None
    return _evict(st)


def _library(st):
    from bit_attention_video_smooth_gb300 import vca
    c = st["case"]
    cache = vca.Cache(st["k8"], st["v8"], st["sk"], st["sv"], st["table"], st["length"])
    if c["op"] == "append":
        return vca.cache_append(cache, st["K"], st["V"], st["start"])
    if c["op"] == "attention":
        return vca.cache_attention(cache, st["Q"], st["start"], causal=c["causal"], softcap=c["softcap"], ws=st["ws"])
    if c["op"] == "weigh":
        return vca.cache_weigh(cache, st["Q"], st["start"], st["lse"], st["weight"], causal=c["causal"],
                               softcap=c["softcap"], ws=st["ws"])
    return vca.cache_evict(cache, st["weight"], st["fresh"], c["budget"], c["recent"], kept=st["kept"])[0]


def run(state):
    out = _library(state) if own else _plain(state)
    op = state["case"]["op"]
    if op == "attention":
        return {"o": out[0], "lse": out[1]}
    if op == "weigh":
        return {"weight": state["weight"]}
    held = {"k": state["k8"].view(torch.float8_e4m3fn), "v": state["v8"].view(torch.float8_e4m3fn),
            "sk": state["sk"], "sv": state["sv"]}
    if op == "evict":
        held.update(length=out, kept=state["kept"], weight=state["weight"])
    return held


# ---------------------------------------------------------------------------
# The definition in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------
def _grid(x):
    """The E4M3 value nearest to each x in 64 bits, ties to even; |x| <= 448."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp_min(-6.0)
    e = torch.where(a >= torch.exp2(e + 1), e + 1, torch.where((a < torch.exp2(e)) & (e > -6), e - 1, e))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _pow2_at_least(a):
    s = SMIN
    e = math.floor(math.log2(max(a / EMAX, SMIN))) - 1
    while math.ldexp(1.0, e) * EMAX < a:
        e += 1
    return max(s, math.ldexp(1.0, e))


def _exact_rows(st, b, h, codes, scale):
    m = int(st["length"][b])
    page = st["table"][b, :-(-m // PAGE)].long()
    x = codes[page, h].view(torch.float8_e4m3fn).double() * scale[page, h].double()[:, None, None]
    return x.reshape(-1, D)[:m], page


def _exact_scores(st, b, h):
    """Scores [n][G][len] of one sequence and KV head in 64 bits and whether each key is visible to each row."""
    c = st["case"]
    G = c["Hq"] // c["Hkv"]
    lo, hi, m = int(st["start"][b]), int(st["start"][b + 1]), int(st["length"][b])
    k, _ = _exact_rows(st, b, h, st["k8"], st["sk"])
    s = torch.matmul(st["Q"][lo:hi, h * G:(h + 1) * G].double(), k.T) / math.sqrt(D)
    if c["softcap"] > 0:
        s = torch.tanh(s / c["softcap"]) * c["softcap"]
    if c["causal"]:
        at = torch.arange(m, device="cuda")
        row = torch.arange(hi - lo, device="cuda") + (m - (hi - lo))
        s.masked_fill_((at > row[:, None])[:, None], -math.inf)
    return s, lo, hi, m, G


def exact(case, seed):
    st = prepare(case, seed)
    news, lens = _lens(case)
    op, B, Hq, Hkv = case["op"], case["B"], case["Hq"], case["Hkv"]
    if op in ("attention", "weigh") and 4 * D * Hq * _visible(case) > 3e12:
        return None
    if op == "attention":
        T = st["Q"].shape[0]
        o = torch.empty((T, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.empty((T, Hq), dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(Hkv):
                s, lo, hi, m, G = _exact_scores(st, b, h)
                z = torch.logsumexp(s, -1)
                v, _ = _exact_rows(st, b, h, st["v8"], st["sv"])
                o[lo:hi, h * G:(h + 1) * G] = torch.exp(s - z[..., None]) @ v
                lse[lo:hi, h * G:(h + 1) * G] = z
        return {"o": o, "lse": lse}
    if op == "weigh":
        w = st["weight"].double()
        for b in range(B):
            for h in range(Hkv):
                s, lo, hi, m, G = _exact_scores(st, b, h)
                got = torch.exp(s - st["lse"][lo:hi, h * G:(h + 1) * G].double()[..., None]).sum((0, 1))
                _, page = _exact_rows(st, b, h, st["k8"], st["sk"])
                flat = w[page, h].reshape(-1)
                flat[:m] += got
                w[page, h] = flat.view(-1, PAGE)
        return {"weight": w}
    out = {"k": st["k8"].view(torch.float8_e4m3fn).double(), "v": st["v8"].view(torch.float8_e4m3fn).double(),
           "sk": st["sk"].double(), "sv": st["sv"].double()}
    if op == "append":
        for x, s, rows in (("k", "sk", "K"), ("v", "sv", "V")):
            X, start = st[rows].double(), st["start"].tolist()
            for b in range(B):
                m, n = lens[b], news[b]
                for col in range((m - n) // PAGE, -(-m // PAGE)):
                    p = int(st["table"][b, col])
                    lo, hi = max(m - n, col * PAGE), min(m, (col + 1) * PAGE)
                    new = X[start[b] + lo - (m - n):start[b] + hi - (m - n)]       # [rows][H][D]
                    a = new.abs().amax((0, 2)).tolist()
                    sc = torch.tensor([_pow2_at_least(v) for v in a], dtype=torch.float64, device="cuda")
                    r = lo - col * PAGE
                    if r > 0:
                        sc = torch.maximum(sc, out[s][p])
                        out[x][p, :, :r] = _grid(out[x][p, :, :r] * (out[s][p] / sc)[:, None, None])
                    out[x][p, :, r:r + hi - lo] = _grid(new.transpose(0, 1) / sc[:, None, None])
                    out[s][p] = sc
        return out
    kept = st["kept"].clone()
    w = st["weight"].double()
    for b in range(B):
        m = lens[b]
        stay, recent = min(m, case["budget"]), min(m, case["recent"])
        for h in range(Hkv):
            k, page = _exact_rows(st, b, h, st["k8"], st["sk"])
            v, _ = _exact_rows(st, b, h, st["v8"], st["sv"])
            wt = st["weight"][page, h].reshape(-1)[:m].double()
            heavy = torch.argsort(-wt[:m - recent], stable=True)[:stay - recent]
            at = torch.cat([heavy.sort().values, torch.arange(m - recent, m, device="cuda")])
            kept[b, h, :stay] = at.to(torch.int32)
            for j in range(0, stay, PAGE):
                p, sel = int(st["fresh"][b, j // PAGE]), at[j:j + PAGE]
                for x, s, val in (("k", "sk", k), ("v", "sv", v)):
                    sc = _pow2_at_least(float(val[sel].abs().max()))
                    out[x][p, h, :sel.numel()] = _grid(val[sel] / sc)
                    out[s][p, h] = sc
                w[p, h, :sel.numel()] = wt[sel]
    out.update(length=None, kept=None, weight=w)
    return out
