"""The hand-offs between the warps of the tensor-memory attention kernel on single tiles, as a
model on the CPU: softmax and issuing warps of both tiles walk over items of one to three
blocks in every order that their barriers allow, and no wait may meet a later phase than the
one it means (a barrier tells two phases in a row apart, not three)."""
import pytest

# arrivals per phase: queries, sums of tile 1, "they have been read", "no round of tile 1",
# and for each tile and round in turn scores, weights, products
COUNT = {"q": 2, "m": 1, "f": 1, "i": 1,
         **{f"{what}{tile}{turn}": 1 for what in "spo" for tile in "01" for turn in "01"}}


def programs(items, idle, rescales):
    """(operation, barrier, phase) of each warp; `items` are numbers of blocks.  `rescales`:
    every round but an item's first waits for the products before it."""
    soft, issue = [[], []], [[], []]
    rounds, idles = [0, 0], 0
    for k, blocks in enumerate(items):
        for x in (0, 1):
            n, r0 = (blocks + 1 - x) // 2, rounds[x]
            name = lambda what, r: f"{what}{x}{r & 1}"  # noqa: E731
            soft[x].append(("arrive", "q", 0))
            for r in range(r0, r0 + n):
                soft[x].append(("wait", name("s", r), r >> 1))
                if rescales and r > r0:
                    soft[x].append(("wait", name("o", r - 1), (r - 1) >> 1))
                soft[x].append(("arrive", name("p", r), 0))
            if n:
                soft[x].append(("wait", name("o", r0 + n - 1), (r0 + n - 1) >> 1))
            issue[x].append(("wait", "q", k))
            issue[x] += [("arrive", name("s", r), 0) for r in range(r0, r0 + min(n, 2))]
            for r in range(r0, r0 + n):
                issue[x] += [("wait", name("p", r), r >> 1), ("arrive", name("o", r), 0)]
                if r + 2 < r0 + n:
                    issue[x].append(("arrive", name("s", r + 2), 0))
            if not n and idle:
                issue[x].append(("arrive", "i", 0))
                soft[x].append(("wait", "i", idles))
                idles += 1
            rounds[x] += n
        soft[1].extend([("arrive", "m", 0), ("wait", "f", k)])
        soft[0].extend([("wait", "m", k), ("arrive", "f", 0)])
    return [*soft, *issue]


def faults(items, idle, rescales=False):
    """Reachable states in which a wait meets the wrong phase or nothing can go on."""
    progs, bars = programs(items, idle, rescales), list(COUNT)
    start = ((0,) * 4, ((0, 0),) * len(bars))
    seen, todo, wrong = {start}, [start], 0
    while todo:
        at, state = todo.pop()
        moved = False
        for w, prog in enumerate(progs):
            if at[w] == len(prog):
                continue
            op, name, phase = prog[at[w]]
            b, after = bars.index(name), list(state)
            done, arrived = state[b]
            if op == "arrive":
                full = arrived + 1 == COUNT[name]
                after[b] = (done + full, 0 if full else arrived + 1)
            elif done % 2 == phase % 2:  # the phase in progress has this parity: it waits
                wrong += done != phase
                continue
            else:
                wrong += done != phase + 1
            moved = True
            step = (tuple(p + (k == w) for k, p in enumerate(at)), tuple(after))
            if step not in seen:
                seen.add(step)
                todo.append(step)
        if not moved and any(p < len(prog) for p, prog in zip(at, progs)):
            wrong += 1
    return wrong


@pytest.mark.parametrize("rescales", [False, True])
@pytest.mark.parametrize("items", [[1] * 6, [1, 2, 1, 1, 3, 1], [5, 1, 1, 1, 4], [3, 1, 2, 1, 1, 7]])
def test_no_wait_meets_a_wrong_phase(items, rescales):
    assert faults(items, idle=True, rescales=rescales) == 0


def test_the_model_sees_an_issuer_that_falls_behind():
    """What the barrier for items without a round is there for."""
    assert faults([1] * 6, idle=False) > 0
    assert faults([2] * 6, idle=False) == 0
