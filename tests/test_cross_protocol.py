"""Discrete-event model of how the forward kernel of the attention to an encoder's states hands
scores, probabilities and finished blocks between its warps (CPU only).

A CTA walks its units one after the other without a barrier between them: the issuing warp, whose
products run in order in the tensor pipe; four softmax warps for each of the blocks A and B; four
output warps. Units of an item without a valid key have no tiles: the issuer passes over them,
the softmax and the output warps do not. Each agent below is one warp with the waits and arrivals
of csrc/cross_fwd.cu in their order; the loaders are left out (their tiles are always there).
Agents run in random order with random speeds, and every read is checked: the scores of the
softmax warp's own tile, the probabilities of the product's own tile, O with exactly the unit's
tiles so far, the 1 / l of the output's own unit.

An mbarrier's test for parity P succeeds when the phase in progress has the other parity, so a
thread that has not seen the phase before the awaited one may pass two phases early. The issuer
that waited for the block before O to be read out ahead of the new unit's probabilities did so
behind units without keys; the model shows it.

The second model is of the elementwise warps of the dq kernel when a bounded wait runs out: the
eight warps meet at barriers that wait without a limit, so whoever gives up has to leave together
with the others.
"""
import os
import random
import re

import pytest

WARPS = 4


class Stale(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passed(self, parity):
        return lambda: (self.phase & 1) != (parity & 1)


def need(ok, what):
    if not ok:
        raise Stale(what)


def run(units, seed, wait_ahead=False):
    """units: (key tiles, has a block B). True if all of them finish, False where the agents wait for
    one another for good; Stale on a wrong read. wait_ahead: the issuer waits for O before the
    unit's probabilities instead of behind them."""
    rng = random.Random(seed)
    two = range(2)
    sfull, odone = [Bar(1) for _ in two], [Bar(1) for _ in two]
    pfull = [[Bar(WARPS) for _ in two] for _ in two]
    lfull, oempty = [Bar(WARPS) for _ in two], [Bar(WARPS) for _ in two]
    s = [[None] * WARPS for _ in two]                       # the tile whose scores a warp's lanes hold
    p = [[[None] * WARPS for _ in two] for _ in two]        # [block][half][warp]
    inv = [[None] * WARPS for _ in two]
    o = [(None, 0) for _ in two]                            # unit, tiles summed
    queue, met = [], [0, 0]                                 # the pipe; arrivals at the output warps' barriers
    free = lambda: True

    def issuer():
        rows, at = [0, 0], [-1]

        def opened():                                       # the next unit with tiles
            while at[0] + 1 < len(units):
                at[0] += 1
                rows[0] += 1
                rows[1] += units[at[0]][1]
                if units[at[0]][0]:
                    return True
            at[0] = len(units)
            return False

        def scores(x, u, t):
            queue.append(("s", x, u, t))
            queue.append(("commit", sfull[x]))

        np_ = [0, 0]
        if not opened():
            return
        u, t = at[0], 0
        for x in range(1 + units[u][1]):
            scores(x, u, t)
        while u < len(units):
            n, has_b = units[u]
            row, nu, nt = list(rows), u, t + 1
            for x in two:
                if x == 0 or has_b:
                    if wait_ahead and t == 0 and row[x] > 1:
                        yield oempty[x].passed(row[x])
                    yield pfull[x][0].passed(np_[x])
                    if not wait_ahead and t == 0 and row[x] > 1:
                        yield oempty[x].passed(row[x])
                    queue.append(("pv", x, u, t, 0))
                    yield pfull[x][1].passed(np_[x])
                    np_[x] += 1
                    queue.append(("pv", x, u, t, 1))
                    if t + 1 == n:
                        queue.append(("commit", odone[x]))
                if x == 0 and nt == n:
                    opened()
                    nu, nt = at[0], 0
                if nu < len(units) and (x == 0 or units[nu][1]):
                    scores(x, nu, nt)
            u, t = nu, nt

    def pipe():
        while True:
            yield lambda: bool(queue)
            op = queue.pop(0)
            if op[0] == "commit":
                op[1].arrive()
                continue
            x, u, t = op[1:4]
            if op[0] == "s":
                s[x] = [(u, t)] * WARPS
                continue
            half = op[4]
            need(all(w == (u, t) for w in p[x][half]), "P V of another tile's probabilities")
            if half == 0:
                need(t == 0 or o[x] == (u, t), "P V onto another unit's sum")
                o[x] = (u, t + 0.5)
            else:
                need(o[x] == (u, t + 0.5), "O overwritten between the halves")
                o[x] = (u, t + 1)

    def softmax(x, w):
        ns = nu = 0
        for u, (n, has_b) in enumerate(units):
            if x and not has_b:
                continue
            for t in range(n):
                yield sfull[x].passed(ns)
                ns += 1
                need(s[x][w] == (u, t), "scores of another tile")
                need(t == 0 or o[x] == (u, t), "a rescale of another sum")
                for half in two:
                    yield free
                    p[x][half][w] = (u, t)
                    pfull[x][half].arrive()
            if nu:
                yield oempty[x].passed(nu - 1)
            nu += 1
            inv[x][w] = u
            lfull[x].arrive()

    def output(w):
        nl, no, mine = [0, 0], [0, 0], 0
        for u, (n, has_b) in enumerate(units):
            for x in range(1 + has_b):
                yield lfull[x].passed(nl[x])
                nl[x] += 1
                if n:
                    yield odone[x].passed(no[x])
                    no[x] += 1
                for step in two:                            # the barriers ahead of and behind the staging
                    met[step] += 1
                    mine += step == 0
                    yield lambda step=step, mine=mine: met[step] >= WARPS * mine
                    if step == 0:
                        yield free
                        need(all(i == u for i in inv[x]), "1 / l of another unit")
                        need(n == 0 or o[x] == (u, n), "O of another unit")
                        oempty[x].arrive()

    agents = [issuer()] + [softmax(x, w) for x in two for w in range(WARPS)] + [output(w) for w in range(WARPS)]
    count = len(agents)
    agents.append(pipe())
    speed = [rng.choice([0.02, 0.2, 1.0]) for _ in agents]
    if rng.random() < 0.5:
        speed[9:13] = [0.02] * WARPS                        # a store that takes long
    conds = [next(a, None) for a in agents]
    while any(conds[:count]):
        ready = [i for i, c in enumerate(conds) if c and c()]
        if not ready:
            return False
        i = rng.choices(ready, [speed[i] for i in ready])[0]
        conds[i] = next(agents[i], None)
    return True


def sequences(seed):
    rng = random.Random(seed)
    yield [(1, True), (1, True), (0, True), (1, True), (1, True), (1, True)]
    yield [(0, True), (1, True), (0, True), (0, True), (2, True), (1, True), (1, False)]
    yield [(0, False)] * 3
    yield [(1, True), (0, True), (0, True), (0, False), (3, True), (0, True), (1, True), (1, True)]
    for _ in range(6):
        yield [(rng.choice([0, 0, 1, 1, 2, 5]), rng.random() < 0.8) for _ in range(rng.randint(1, 12))]


@pytest.mark.parametrize("seed", range(60))
def test_every_read_sees_its_own_unit(seed):
    for i, units in enumerate(sequences(seed)):
        assert run(units, 100 * seed + i), units


def test_waiting_for_o_ahead_of_the_probabilities_is_caught():
    caught = 0
    for seed in range(400):
        try:
            caught += not run([(1, True), (1, True), (0, True), (1, True), (1, True), (1, True)], seed, wait_ahead=True)
        except Stale:
            caught += 1
    assert caught


DQ_WARPS = 8


def run_dq_give_up(units, seed, leave_alone=False):
    """units: key tiles. The products stop at a random point, and some time later a wait elsewhere
    runs out; each warp sees that at its own time. True if all warps leave. leave_alone: a warp
    whose wait ran out goes without a word."""
    rng = random.Random(seed)
    phases = [("s", "t")] * sum(units)
    last = rng.randint(0, 2 * len(phases))                  # products that are still done
    done = {"s": 0, "t": 0, "out": 0}
    abort = [False]
    met, votes = [0], {}

    def barrier(mine, vote):                                # of all warps; whether all said yes
        votes[mine] = votes.get(mine, True) and vote
        met[0] += 1
        return lambda: met[0] >= DQ_WARPS * (mine + 1)

    def warp():
        n = {"s": 0, "t": 0, "out": 0}
        gen, held = 0, False

        def reached(kind):
            # as wait_phase: the phase first, then the flag
            return lambda: done[kind] > n[kind] or abort[0]

        def taken(kind):
            ok = done[kind] > n[kind]
            n[kind] += 1
            return ok

        for tiles in units + [None]:
            if not tiles:                                   # no keys, or the end
                steps = (["out"] if held else []) + (["empty"] if tiles == 0 else [])
                held = False
            else:
                steps = []
                for i in range(tiles):
                    steps += ["s"] + (["out"] if held else []) + ["t"]
                    held = False
                held = True
            for step in steps:
                ok = True
                if step != "empty":
                    yield reached(step)
                    ok = taken(step)
                if step in ("out", "empty") or (step == "t" and tiles == 1):
                    yield barrier(gen, ok)
                    ok, gen = votes[gen], gen + 1
                    if not ok:
                        return
                    if step != "t":
                        yield barrier(gen, True)
                        gen += 1
                elif not ok:
                    if not leave_alone:
                        yield barrier(gen, False)
                    return

    def products():
        for i in range(last):
            done["s" if i % 2 == 0 else "t"] += 1
            done["out"] = sum(done["t"] >= sum(units[:u + 1]) for u in range(len(units)) if units[u])
            yield lambda: True

    def clock():
        for _ in range(rng.randint(0, 60)):
            yield lambda: True
        abort[0] = True

    agents = [warp() for _ in range(DQ_WARPS)] + [products(), clock()]
    conds = [next(a, None) for a in agents]
    while any(conds[:DQ_WARPS]):
        ready = [i for i, c in enumerate(conds) if c and c()]
        if not ready:
            return False
        i = rng.choice(ready)
        conds[i] = next(agents[i], None)
    return True


DQ_UNITS = [[1], [2], [3, 1, 0, 2], [1, 1, 1], [0, 2, 2], [4, 4], [0, 0]]


@pytest.mark.parametrize("units", DQ_UNITS, ids=str)
def test_dq_warps_leave_together(units):
    assert all(run_dq_give_up(units, seed) for seed in range(500))


def test_a_dq_warp_that_leaves_alone_is_caught():
    for units in ([3, 1, 0, 2], [4, 4], [2]):
        assert not all(run_dq_give_up(units, seed, leave_alone=True) for seed in range(2000))


def test_warps_converge_ahead_of_reads_of_tmem():
    """tcgen05.ld takes whole converged warps. In loops that are not unrolled the read follows the
    stores of the turn before, which lanes without a row or key of their own skip: each such
    loop begins with a __syncwarp, and no turn is cut short for some lanes."""
    here = os.path.join(os.path.dirname(__file__), "..", "block_sparse_attention_major_b200", "csrc")
    loops = 0
    for name in ("cross_fwd.cu", "cross_bwd.cu"):
        with open(os.path.join(here, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"#pragma unroll 1\s+for \([^{]*\) \{", text):
            depth, at = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            body = text[m.end():at]
            if "tmem_ld" not in body or "warp_wait" in body:
                continue                    # a loop over whole blocks: its waits are votes of the warp
            loops += 1
            assert body.split()[0] == "__syncwarp();", (name, m.group(0))
            assert not re.search(r"if \(key[^)]*\) continue", body), name
    assert loops == 4
