"""Model check of the mbarrier protocol of the tcgen05 attention over the 8-bit cache (csrc/cache_tc.cu), run on the CPU
with the engine of test_bwd_protocol.

Agents: the TMA warp (codes of K and V, and a ring of four scale records), the converter warps (one agent: they move in
step through their barriers), the MMA warp, and three pairs of softmax agents (the two halves of a lane quarter), one pair
of them without rows.  Besides deadlock and the parity rule (a wait for phase k must see k or k + 1 completed phases), these data hazards are
checked: codes overwritten before they are converted, scale records before every reader has them, fp16 tiles before
the MMA that reads them is done, score buffers before their P is used, and O rescaled under a PV."""
import random
from collections import defaultdict

import pytest

from test_bwd_protocol import run_agents

TILE_COUNTS = [1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 16, 33]
PAIRS = 3  # lane quarters modelled; the last has no rows


def simulate(n, rng, drop=None):
    """drop: a wait to leave out (negative controls)."""
    need = defaultdict(lambda: 1)
    need.update({f"p_full{x}": 2 * PAIRS for x in range(2)})
    need.update({f"i_empty{x}": 2 * PAIRS for x in range(4)})
    for q in range(PAIRS):
        for j in range(n + 1):
            need[f"pair{q}_{j}"] = 2
    count, done, hazards = defaultdict(int), defaultdict(int), []
    seen = defaultdict(int)  # progress that the hazards are judged by

    def arrive(b):
        count[b] += 1
        if count[b] == need[b]:
            count[b] = 0
            done[b] += 1

    def wait(b, k):
        if drop != b.rstrip("0123456789"):
            yield ("wait", b, k)

    def tma():
        for j in range(n):
            for kv in "kv":
                if j >= 1:
                    yield from wait(f"c_empty_{kv}", j - 1)
                if seen["conv_" + kv] < j:
                    hazards.append(("tma", f"codes of {kv}{j - 1} overwritten", j))
                yield ("arrive", f"c_full_{kv}")
                if kv == "k":
                    if j >= 4:
                        yield from wait(f"i_empty{j & 3}", (j >> 2) - 1)
                    late = [w for w in ["conv_v"] + [f"soft{q}{h}" for q in range(PAIRS) for h in range(2)] if seen[w] < j - 3]
                    if late:
                        hazards.append(("tma", f"scales of {j - 4} overwritten", late))
                    yield ("arrive", f"i_full{j & 3}")

    def conv():
        yield ("arrive", "q_full")
        for j in range(n):
            x = j & 1
            for kv in "kv":
                yield from wait(f"c_full_{kv}", j)
                if j >= 2:
                    yield from wait(f"{kv}_empty{x}", (j >> 1) - 1)
                if seen["mma_" + kv] < j - 1:
                    hazards.append(("conv", f"{kv} tile {j - 2} overwritten", j))
                if kv == "v":
                    yield from wait(f"i_full{j & 3}", j >> 2)
                seen["conv_" + kv] = j + 1
                yield ("arrive", f"c_empty_{kv}")
                yield ("arrive", f"{kv}_full{x}")

    def mma():
        yield ("wait", "q_full", 0)
        for j in range(n + 1):
            if j < n:
                x = j & 1
                yield from wait(f"k_full{x}", j >> 1)
                if j >= 2 and done[f"p_full{x}"] < (j >> 1):
                    hazards.append(("mma", f"S{j} over P{j - 2}", j))
                seen["mma_k"] = j + 1
                yield ("arrive", f"s_full{x}")
                yield ("arrive", f"k_empty{x}")
            if j >= 1:
                jj, x = j - 1, (j - 1) & 1
                yield from wait(f"v_full{x}", jj >> 1)
                yield from wait(f"p_full{x}", jj >> 1)
                if seen["conv_v"] < j:
                    hazards.append(("mma", f"PV{jj} before V", j))
                seen["mma_v"] = j
                yield ("arrive", f"v_empty{x}")
                yield ("arrive", "o_done")

    def softmax(q, half):
        active = q < PAIRS - 1
        yield ("wait", "q_full", 0)
        for j in range(n):
            yield from wait(f"i_full{j & 3}", j >> 2)
            seen[f"soft{q}{half}"] = j + 1
            yield ("arrive", f"i_empty{j & 3}")
            yield from wait(f"s_full{j & 1}", j >> 1)
            if active:
                yield ("arrive", f"pair{q}_{j}")
                yield ("wait", f"pair{q}_{j}", 0)
                if j >= 1:
                    yield from wait("o_done", j - 1)
                    if done["o_done"] != j:
                        hazards.append(("softmax", "O rescaled under a PV", j))
            yield ("arrive", f"p_full{j & 1}")
        if active:
            yield ("wait", "o_done", n - 1)

    agents = {"tma": tma(), "conv": conv(), "mma": mma()}
    agents.update({f"softmax{q}{h}": softmax(q, h) for q in range(PAIRS) for h in range(2)})
    return run_agents(agents, arrive, done, hazards, rng)


def test_protocol_never_deadlocks_aliases_or_races():
    rng = random.Random(4)
    for trial in range(600):
        n = TILE_COUNTS[trial % len(TILE_COUNTS)]
        finished, hazards = simulate(n, rng)
        assert finished and not hazards, (n, hazards[:3])


# (The wait on i_empty follows from the others: V_{j-2} is converted after PV_{j-4}, so after the softmax has read scales j - 4.)
@pytest.mark.parametrize("drop,n,trials", [("c_empty_v", 16, 300), ("k_empty", 16, 300), ("v_empty", 16, 300), ("v_full", 1, 20000),
                                           ("p_full", 16, 300), ("o_done", 16, 300)])
def test_model_flags_a_missing_wait(drop, n, trials):
    rng = random.Random(5)
    for _ in range(trials):
        finished, hazards = simulate(n, rng, drop=drop)
        if hazards or not finished:
            return
    raise AssertionError(drop)
