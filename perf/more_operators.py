"""Prompt attention and the cache's page planning as measured workloads.

prompt   attention of packed prompts over their own keys and values, bf16, before these are quantised
         into the cache: Q [T][Hq][128], K, V [T][Hkv][128], the rows start[b] .. start[b+1]-1 are sequence
         b's.  Optionally joined with an attention over what came before: `prior` O and lse.
plan     the step's new tokens get their places: pages for table columns that begin, lengths, the cut of
         the rows, and every row's slot (page * 128 + place in the page) and position.  Free is a page
         that no live table entry names; the lowest free pages go to the sequences in order.
fresh    fresh pages for an eviction to `budget` tokens: ceil(min(length, budget) / 128) a sequence.

`run` computes an operator in elementary torch operations where `own` is false and by the library's entry
points where it is true; `exact` computes the attention in 64 bits and the pages from the definition.
"""
import math

import torch

own = False

D = 128
PAGE = 128


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _prompt(name, B, Hq, Hkv, n, ragged=False, causal=True, softcap=0.0, strided=False, prior=False):
    c = {"op": "prompt", "B": B, "Hq": Hq, "Hkv": Hkv, "n": n, "ragged": ragged, "causal": causal, "softcap": softcap,
         "strided": strided, "prior": prior}
    return {"name": name, **c} if name else c


def _pages(name, op, B, held, new=0, every=1, budget=0):
    """`every`: each `every`-th sequence gets `new` tokens, the others one (with every > 1 the former are
    prompts of sequences that hold nothing yet); budget: that of fresh pages."""
    c = {"op": op, "B": B, "held": held, "new": new, "every": every, "budget": budget}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one question of a few words: latency
        _prompt("prompt_short", 1, 24, 24, 45),
        # a batch of ordinary prompts, five query heads to a KV head
        _prompt("prompt_batch", 32, 40, 8, 1000, ragged=True),
        # prompts of different lengths, capped scores, views of a fused projection
        _prompt("prompt_capped", 4, 32, 8, 2900, ragged=True, softcap=30.0, strided=True),
        # one long document
        _prompt("prompt_long", 1, 40, 8, 32768),
        # a quarter of the 70,656-token video attends to itself, both ways
        _prompt("prompt_frames", 1, 8, 8, 17664, causal=False, strided=True),
        # chunks of sequences whose earlier tokens lie in the cache: joined with the attention over those
        _prompt("prompt_behind_prefix", 8, 40, 8, 2000, ragged=True, prior=True),
        # the decode step: one token each, few begin a page
        _pages("plan_token", "plan", 32, 32768, new=1),
        # decode steps of many short sequences with a prompt among every eight
        _pages("plan_mixed", "plan", 512, 4000, new=700, every=8),
        # a quarter of the 70,656-token video arrives behind what is held
        _pages("plan_chunk", "plan", 1, 40001, new=17664),
        # thousands of sequences, one token each
        _pages("plan_many", "plan", 4096, 2000, new=1),
        # fresh pages for short histories cut to a few hundred tokens
        _pages("fresh_short", "fresh", 2, 1000, budget=300),
        # fresh pages for long prompts cut to an eighth
        _pages("fresh_prompts", "fresh", 64, 32768, budget=4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "plan", "plan", "fresh"])
    if op == "prompt":
        Hq, Hkv = rng.choice([(8, 8), (24, 24), (40, 40), (40, 8), (32, 8), (16, 1), (12, 4), (7, 1)])
        n = _log_int(rng, 1, 16000)
        B = _log_int(rng, 1, max(1, min(64, 3000000 // (n * Hq), 10000000000 // (n * n * Hq))))
        return _prompt("", B, Hq, Hkv, n, ragged=rng.random() < 0.7, causal=rng.random() < 0.7,
                       softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), strided=rng.random() < 0.5, prior=rng.random() < 0.3)
    B = _log_int(rng, 1, 4096)
    held = _log_int(rng, 1, max(1, min(100000, 8000000 // B)))
    if op == "fresh":
        return _pages("", op, B, held, budget=_log_int(rng, 1, held))
    every = rng.choice([1, 2, 8, 64])
    return _pages("", op, B, held, new=_log_int(rng, 1, max(1, min(20000, 100000 * every // B))), every=every)


def _spread(case, most, seed):
    """A number for each sequence, spread evenly from a tenth of the most to all of it."""
    return [max(1, int(most * (1.0 - 0.9 * ((b * seed) % 1.0)))) for b in range(case["B"])]


def _rows(case):
    """New rows of each sequence."""
    if case["op"] == "prompt":
        return _spread(case, case["n"], 0.4142135623730951) if case["ragged"] else [case["n"]] * case["B"]
    many = _spread(case, case["new"], 0.4142135623730951)
    return [many[b] if b % case["every"] == 0 else 1 for b in range(case["B"])]


def _held(case):
    held = _spread(case, case["held"], 0.6180339887498949)
    return [0 if case["every"] > 1 and b % case["every"] == 0 else m for b, m in enumerate(held)]


def _up(n):
    return -(-n // PAGE)


def work(case):
    B = case["B"]
    if case["op"] == "prompt":
        rows, Hq, Hkv = _rows(case), case["Hq"], case["Hkv"]
        T = sum(rows)
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in rows)
        joined = T * Hq * (2 * D + 4) if case["prior"] else 0
        return {"bytes": T * (4 * D * Hq + 4 * D * Hkv + 4 * Hq) + joined + 4 * (B + 1), "flops": 4 * D * Hq * pairs}
    held = _held(case)
    live = sum(_up(m) for m in held)
    if case["op"] == "fresh":
        fresh = sum(_up(min(m, case["budget"])) for m in held)
        return {"bytes": 4 * (B + live + fresh), "flops": live + fresh}
    rows = _rows(case)
    fresh = sum(_up(m + n) - _up(m) for m, n in zip(held, rows))
    return {"bytes": 4 * (4 * B + 1 + (live if fresh else 0) + fresh + 2 * sum(rows)), "flops": 2 * (B + sum(rows))}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _tensor(g, T, H, strided, outliers):
    """bf16 [T][H][128] ~ N(0, 1), four channels a head eight times as large where `outliers`; a view into wider rows where strided."""
    x = torch.randn((T, H + 2 if strided else H, D), generator=g, device="cuda")
    if outliers:
        x = x * torch.where(torch.rand((1, x.shape[1], D), generator=g, device="cuda") < 4 / D, 8.0, 1.0)
    x = x.to(torch.bfloat16)
    return x[:, 1:H + 1] if strided else x


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B = case["B"]
    st = {"case": dict(case)}
    if case["op"] == "prompt":
        rows = _rows(case)
        T, Hq, Hkv = sum(rows), case["Hq"], case["Hkv"]
        st["start"] = _ints([sum(rows[:b]) for b in range(B + 1)])
        st["Q"] = _tensor(g, T, Hq, case["strided"], True)
        st["K"] = _tensor(g, T, Hkv, case["strided"], True)
        st["V"] = _tensor(g, T, Hkv, case["strided"], False)
        if case["prior"]:
            # outputs over a prefix of unit-variance values, some of whose rows saw nothing
            lse = torch.randn((T, Hq), generator=g, device="cuda") * 2.0 + 8.0
            nothing = torch.rand((T, Hq), generator=g, device="cuda") < 0.05
            o = torch.randn((T, Hq, D), generator=g, device="cuda") * 0.2
            st["prior_o"] = torch.where(nothing[..., None], 0.0, o).to(torch.bfloat16)
            st["prior_lse"] = torch.where(nothing, -math.inf, lse)
        return st
    # a pool in use: pages in no order, some free ones among them, the table's columns behind a sequence's last page empty
    held, fresh = _held(case), case["op"] == "fresh"
    rows = [0] * B if fresh else _rows(case)
    live = [_up(m) for m in held]
    need = sum(_up(min(m, case["budget"])) for m in held) if fresh else sum(_up(m + n) - _up(m) for m, n in zip(held, rows))
    pages = sum(live) + need + max(16, (sum(live) + need) // 8)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    cols = max(_up(m + n) for m, n in zip(held, rows)) + 1
    first = _ints([sum(live[:b]) for b in range(B)])
    at = torch.arange(cols, device="cuda")
    named = at < _ints(live)[:, None]
    st["table"] = torch.where(named, order[torch.where(named, first[:, None] + at, 0)], -1).to(torch.int32)
    st["held"] = _ints(held)
    st["pages"] = pages
    # one layer's codes and scales: the plan takes their shape alone
    st["codes"] = torch.zeros((pages, 1, 1, 1), dtype=torch.uint8, device="cuda").expand(pages, 1, PAGE, D)
    st["scales"] = torch.zeros((pages, 1), device="cuda")
    if fresh:
        st["fresh"] = torch.full((B, _up(case["budget"])), -1, dtype=torch.int32, device="cuda")
        return st
    st["new"], st["T"] = _ints(rows), sum(rows)
    st["length"] = st["held"].clone()
    st["slot"] = torch.full((st["T"],), -1, dtype=torch.int32, device="cuda")
    st["position"] = torch.full((st["T"],), -1, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _attend(st):
    c = st["case"]
    Hq, Hkv, G = c["Hq"], c["Hkv"], c["Hq"] // c["Hkv"]
    T = st["Q"].shape[0]
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, Hq), device="cuda")
    lo = 0
    for n in _rows(c):
        hi = lo + n
        step = max(1, (1 << 30) // (G * n * n))                        # KV heads at a time: 4 GB of scores
        for h0 in range(0, Hkv, step):
            h1 = min(Hkv, h0 + step)
            q = st["Q"][lo:hi, h0 * G:h1 * G].float().transpose(0, 1).reshape(h1 - h0, G * n, D)
            k = st["K"][lo:hi, h0:h1].float().permute(1, 2, 0)
            s = torch.matmul(q, k).view(h1 - h0, G, n, n) * (1.0 / math.sqrt(D))
            if c["softcap"] > 0:
                s = c["softcap"] * torch.tanh(s / c["softcap"])
            if c["causal"]:
                at = torch.arange(n, device="cuda")
                s.masked_fill_(at > at[:, None], -math.inf)
            m = s.amax(-1, keepdim=True)
            if c["prior"]:
                before = st["prior_lse"][lo:hi, h0 * G:h1 * G].transpose(0, 1).reshape(h1 - h0, G, n, 1)
                m = torch.maximum(m, before)
            p = torch.exp(s - m)
            del s
            l = p.sum(-1, keepdim=True)
            v = st["V"][lo:hi, h0:h1].float().transpose(0, 1)
            o = torch.matmul(p.view(h1 - h0, G * n, n), v).view(h1 - h0, G, n, D)
            if c["prior"]:
                w = torch.exp(before - m)
                l = l + w
                o = o + w * st["prior_o"][lo:hi, h0 * G:h1 * G].float().transpose(0, 1).reshape(o.shape)
            o = (o / l).reshape((h1 - h0) * G, n, D).transpose(0, 1)
            out[lo:hi, h0 * G:h1 * G] = o.to(torch.bfloat16)
            lse[lo:hi, h0 * G:h1 * G] = (torch.log(l) + m).reshape((h1 - h0) * G, n).transpose(0, 1)
        lo = hi
    return out, lse


def _free_pages(st):
    """Every page, the free ones first and in order."""
    table, live = st["table"], (st["held"].long() + PAGE - 1) // PAGE
    at = torch.arange(table.shape[1], device="cuda")
    named = torch.where(at < live[:, None], table.long(), st["pages"]).reshape(-1)
    used = torch.zeros(st["pages"] + 1, dtype=torch.bool, device="cuda")
    used[named] = True
    return torch.sort(used[:-1].to(torch.uint8), stable=True).indices, live


def _hand_out(table, free, first, many):
    """The next free pages in the columns first .. first + many - 1 of every sequence, in order."""
    before = torch.cumsum(many, 0) - many
    at = torch.arange(table.shape[1], device="cuda")
    new = (at >= first[:, None]) & (at < (first + many)[:, None])
    rank = (before - first)[:, None] + at
    table.copy_(torch.where(new, free[torch.where(new, rank, 0)], table.long()))


def _plan(st):
    held, new = st["held"].long(), st["new"].long()
    free, live = _free_pages(st)
    length = held + new
    _hand_out(st["table"], free, live, (length + PAGE - 1) // PAGE - live)
    st["length"].copy_(length)
    start = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    t = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    at = held[b] + t - start[b]
    st["position"].copy_(at)
    st["slot"].copy_(st["table"][b, at // PAGE].long() * PAGE + at % PAGE)
    return start.to(torch.int32)


def _fresh(st):
    free, _ = _free_pages(st)
    want = torch.clamp(st["held"].long(), max=st["case"]["budget"])
    _hand_out(st["fresh"], free, torch.zeros_like(want), (want + PAGE - 1) // PAGE)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _cache(vca, st, length):
    return vca.Cache(st["codes"], st["codes"], st["scales"], st["scales"], st["table"], length)


def run(state):
    c = state["case"]
    if own:
        from bit_attention_video_smooth_gb300 import vca
    if c["op"] == "prompt":
        if own:
            prior = (state["prior_o"], state["prior_lse"]) if c["prior"] else None
            o, lse = vca.prompt_attention(state["Q"], state["K"], state["V"], state["start"], causal=c["causal"],
                                          softcap=c["softcap"], prior=prior)
        else:
            o, lse = _attend(state)
        return {"o": o, "lse": lse}
    if c["op"] == "fresh":
        if own:
            vca.cache_fresh(_cache(vca, state, state["held"]), c["budget"], out=state["fresh"])
        else:
            _fresh(state)
        return {"fresh": state["fresh"]}
    if own:
        start = vca.cache_plan(_cache(vca, state, state["length"]), state["new"], state["T"], held=state["held"],
                               slot=state["slot"], position=state["position"])[0]
    else:
        start = _plan(state)
    return {"table": state["table"], "length": state["length"], "start": start, "slot": state["slot"],
            "position": state["position"]}


# ---------------------------------------------------------------------------
# The definition, one sequence at a time: attention by query heads in 64 bits, pages on the host
# ---------------------------------------------------------------------------
def _exact_pages(case, seed):
    st = prepare(case, seed)
    held, table = st["held"].tolist(), st["table"].tolist()
    named = {p for m, row in zip(held, table) for p in row[:_up(m)]}
    free = iter(sorted(set(range(st["pages"])) - named))
    if case["op"] == "fresh":
        fresh = st["fresh"].tolist()
        for m, row in zip(held, fresh):
            for j in range(_up(min(m, case["budget"]))):
                row[j] = next(free)
        return {"fresh": _ints(fresh)}
    start, slot, position = [0], [], []
    for m, n, row in zip(held, st["new"].tolist(), table):
        for j in range(_up(m), _up(m + n)):
            row[j] = next(free)
        start.append(start[-1] + n)
        position += range(m, m + n)
        slot += [row[i // PAGE] * PAGE + i % PAGE for i in range(m, m + n)]
    return {"table": _ints(table), "length": _ints([m + n for m, n in zip(held, st["new"].tolist())]), "start": _ints(start),
            "slot": _ints(slot), "position": _ints(position)}


def exact(case, seed):
    if case["op"] != "prompt":
        return _exact_pages(case, seed)
    rows, Hq = _rows(case), case["Hq"]
    if 4 * D * Hq * sum(n * n for n in rows) > 3e12:
        return None
    st = prepare(case, seed)
    G = Hq // case["Hkv"]
    O = torch.empty((sum(rows), Hq, D), dtype=torch.float64, device="cuda")
    Z = torch.empty((sum(rows), Hq), dtype=torch.float64, device="cuda")
    end = 0
    for n in rows:
        this = slice(end, end + n)
        end += n
        hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1) if case["causal"] else None
        for h in range(Hq):
            s = st["Q"][this, h].double() @ st["K"][this, h // G].double().T / math.sqrt(D)
            if case["softcap"] > 0:
                s = torch.tanh(s / case["softcap"]) * case["softcap"]
            if hidden is not None:
                s = s.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(s, -1)
            o = torch.exp(s - z[:, None]) @ st["V"][this, h // G].double()
            if case["prior"]:
                before = st["prior_lse"][this, h].double()
                both = torch.logaddexp(z, before)
                o = torch.exp(z - both)[:, None] * o + torch.exp(before - both)[:, None] * st["prior_o"][this, h].double()
                z = both
            O[this, h], Z[this, h] = o, z
    return {"o": O, "lse": Z}
