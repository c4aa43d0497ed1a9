"""A model of how the prompt kernel's tiles go from one work to the next, searched through on the CPU.

A tile's roles, work by work, each of one key block (the shortest, where the roles
can be furthest apart):
  issuer     waits for all warps' probabilities, and for the epilogue to have read O of the work
             before; then the tensor core completes O (an arrival on o_full) and, in the order of
             issue, the scores of the next work (s_full)
  softmax    each warp: waits for the scores, hands over its probabilities (p_full), writes its rows'
             statistics into the buffer of this turn and arrives on o_full
  epilogue   waits for o_full, reads all warps' statistics of this turn, frees O (o_free)
On every schedule the epilogue must read the statistics of its own work, and all roles must end.
The number of o_full barriers that a tile's works take in turn is the kernel's own.
"""
import pytest

from test_prompt_layout import _constants

WORKS = 5


class Barrier:
    """(arrivals that are missing, phases done) of a barrier of `count` arrivals."""

    def __init__(self, count):
        self.count, self.start = count, (count, 0)

    def arrive(self, state):
        left, done = state
        return (self.count, done + 1) if left == 1 else (left - 1, done)

    @staticmethod
    def passes(state, parity):      # of a phase that is done, until the next one is
        return state[1] % 2 != parity


def search(warps, turns):
    """Every state that can be reached; returns the first fault or None."""
    bars = {"s_full": Barrier(1), "p_full": Barrier(warps), "o_free": Barrier(1)}
    bars.update({f"o_full{i}": Barrier(1 + warps) for i in range(turns)})
    names = list(bars)
    at = {n: i for i, n in enumerate(names)}

    def o_full(k):
        return f"o_full{k % turns}", (k // turns) & 1

    # what a role does step by step: (wait, barrier, parity), (arrive, barrier) or (stats, work)
    issuer = []
    for k in range(WORKS):
        issuer.append(("wait", "p_full", k & 1))
        if k:
            issuer.append(("wait", "o_free", (k - 1) & 1))
        issuer.append(("issue", k))
    tensor = [("arrive", "s_full")]
    for k in range(WORKS):
        tensor += [("issued", k), ("arrive", o_full(k)[0]), ("arrive", "s_full")]
    softmax, epilogue = [], []
    for k in range(WORKS):
        softmax += [("wait", "s_full", k & 1), ("arrive", "p_full"), ("write", k), ("arrive", o_full(k)[0])]
        epilogue += [("wait", *o_full(k)), ("read", k), ("arrive", "o_free")]
    roles = [issuer, tensor, epilogue] + [softmax] * warps

    first = ((0,) * len(roles), tuple(b.start for b in bars.values()), ((-1, -1),) * warps, -1)
    seen, todo = {first}, [first]
    while todo:
        pcs, state, stats, issued = todo.pop()
        moved = False
        for r, role in enumerate(roles):
            if pcs[r] == len(role):
                continue
            op, *arg = role[pcs[r]]
            new_state, new_stats, new_issued = state, stats, issued
            if op == "wait":
                if not Barrier.passes(state[at[arg[0]]], arg[1]):
                    continue
            elif op == "issued":
                if issued < arg[0]:
                    continue
            elif op == "issue":
                new_issued = arg[0]
            elif op == "arrive":
                i = at[arg[0]]
                new_state = state[:i] + (bars[arg[0]].arrive(state[i]),) + state[i + 1:]
            elif op == "write":
                w, k = r - 3, arg[0]
                new_stats = stats[:w] + (tuple(k if i == k % 2 else x for i, x in enumerate(stats[w])),) + stats[w + 1:]
            elif op == "read":
                if any(x[arg[0] % 2] != arg[0] for x in stats):
                    return f"work {arg[0]}: statistics of works {[x[arg[0] % 2] for x in stats]}"
            moved = True
            nxt = (pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], new_state, new_stats, new_issued)
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
        if not moved and any(pc < len(role) for pc, role in zip(pcs, roles)):
            return f"no role goes on: {pcs}"
    return None


@pytest.mark.parametrize("warps", [2, 3, 4])
def test_the_epilogue_reads_its_own_works_statistics(warps):
    assert search(warps, _constants()[0].get("kTurns", 1)) is None


def test_one_barrier_for_all_works_is_not_enough():
    """A warp that is a work ahead arrives in the place of one that has handed over its probabilities, not its statistics."""
    assert "statistics" in search(2, 1)
