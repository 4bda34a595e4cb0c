"""A discrete model of the hand-offs of the distillation kernel's persistent
blocks, run on the CPU over many random interleavings, in which waits may run
out at any point.

A cluster of blocks takes rows together; a block has computing warps and one
warp that works ahead (the kernel's comment lists their barriers).  Barriers
count as mbarriers do (arrivals and bytes; a wait is by phase parity), and
copies and stores to other blocks land at any later time.  Checked:

  - a wait never passes early: what it stands for is there, for the right row;
  - nothing is overwritten while it may be read;
  - every warp ends, and nothing lands in a block that has gone;
  - a row whose loss is not NaN is whole in every block.

The model finds the faults of blocks that go on after a wait ran out.
"""

import random

import pytest

SETS, GW = 4, 2


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.done = count, count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.pending, self.done = self.count, self.done + 1

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than the phase has"
        self.tx += tx
        self.pending -= 1
        self._turn()

    def land(self, tx):
        self.tx -= tx
        self._turn()

    def passes(self, phase):
        return (self.done & 1) != (phase & 1)


class Block:
    def __init__(self):
        self.full, self.summed, self.listed, self.empty = Bar(1), Bar(GW), Bar(1), Bar(GW)
        self.xch, self.parts = [Bar(1) for _ in range(SETS)], [Bar(1) for _ in range(SETS)]
        self.pairs = [{} for _ in range(SETS)]     # (block, warp) -> row
        self.loss_parts = [{} for _ in range(SETS)]
        self.buf = None                            # row in the buffer
        self.readers = 0                           # warps that may still read it
        self.gave_up = False
        self.gone = 0                              # warps that have exited
        self.sent = {}
        self.dense, self.listed_out = {}, set()    # rows' stores


class Fault(AssertionError):
    pass


def need(ok, what):
    if not ok:
        raise Fault(what)


def run(C, grad, weights, seed, lose, sound=True):
    """One interleaving.  `lose`: the chance that a wait which is not over at a
    look runs out.  Returns the number of rows marked as not whole."""
    rng = random.Random(seed)
    rows = len(weights)
    learn = [rng.random() < 0.8 for _ in range(rows)]
    blocks = [Block() for _ in range(C)]
    loss = [None] * rows
    flying = []                                    # (block, act)
    meet = {"n": 0, "turn": 0}
    everyone = C * (GW + 1)

    def wait(r, bar, phase):
        while True:
            if bar.passes(phase):
                return True
            if sound and blocks[r].gave_up or rng.random() < lose:
                blocks[r].gave_up = True
                return False if sound else True    # the unsound form goes on
            yield

    def barrier():
        turn = meet["turn"]
        meet["n"] += 1
        if meet["n"] == everyone:
            meet["n"], meet["turn"] = 0, turn + 1
        while meet["turn"] == turn:
            yield

    def send(to, bar, act):
        def land():
            act()
            bar.land(8)
        flying.append((to, land))

    def send_pairs(r, k, n, row):
        b = n % SETS
        if k == 0:
            blocks[r].xch[b].arrive(8 * GW * C)
        for to in range(C):
            send(to, blocks[to].xch[b], lambda to=to: blocks[to].pairs[b].__setitem__((r, k), row))

    def send_part(r, n, row):
        b = n % SETS
        if r == 0:
            blocks[0].parts[b].arrive(8 * C)
        send(0, blocks[0].parts[b], lambda: blocks[0].loss_parts[b].__setitem__(r, row))

    def fetch(r, row):
        B = blocks[r]
        need(B.readers == 0, "a copy is started over a row that may be read")
        B.full.arrive(16)

        def land():
            B.buf, B.readers = row, GW + 1
            B.full.land(16)
        flying.append((r, land))

    def leave(r, k, row, sent, fetched):
        B = blocks[r]
        if row < rows:
            for x in blocks:
                x.gave_up = True
        yield from barrier()
        if not any(x.gave_up for x in blocks):
            return
        need(B.gave_up, "the blocks differ on whether one gave up")
        if C > 1:
            B.sent[k] = sent
            yield from barrier()
            most = max(x.sent[j] for x in blocks for j in ([GW] if k == GW else range(GW)))
            need(most - sent <= 2, "more than two rows behind")
            while sent < most:
                if k == GW:
                    send_part(r, sent, -1)
                else:
                    send_pairs(r, k, sent, -1)
                sent += 1
            yield from barrier()
            if k == 0 or (k == GW and r == 0):
                for n in range(max(most - SETS, 0), most):
                    bar = (B.parts if k == GW else B.xch)[n % SETS]
                    while not bar.passes(n // SETS):
                        yield
        if k == GW:
            while fetched and not B.full.passes(fetched - 1):
                yield
            for x in range(row, rows):
                loss[x] = "nan"

    def ahead(r):
        B = blocks[r]
        row = e = sent = fetched = 0
        early = False
        if weights[0]:
            fetch(r, 0)
            fetched += 1
            B.listed.arrive()
        while row < rows and not early:
            more = row + 1 < rows and weights[row + 1]
            if weights[row]:
                early = True               # until the row is over
                if not (yield from wait(r, B.full, e)):
                    break
                need(B.buf == row or not sound, "the ahead warp reads another row")
                if not (yield from wait(r, B.summed, e)):
                    break
                if not grad:
                    B.readers -= 1 if sound else B.readers
                    if more:
                        fetch(r, row + 1)
                        fetched += 1
                if C > 1 and not (yield from wait(r, B.xch[e % SETS], e // SETS)):
                    break
                if C > 1:
                    got = B.pairs[e % SETS]
                    need(len(got) == GW * C and all(x == row for x in got.values()), "pairs of another row")
                    send_part(r, e, row)
                    sent = e + 1
                    if r == 0:
                        if not (yield from wait(r, B.parts[e % SETS], e // SETS)):
                            break
                        need(all(B.loss_parts[e % SETS].get(x) == row for x in range(C)), "parts of another row")
                if r == 0:
                    loss[row] = "value"
                yield
                if grad:
                    if not (yield from wait(r, B.empty, e)):
                        break
                    B.readers -= 1 if sound else B.readers
                    if more:
                        fetch(r, row + 1)
                        fetched += 1
                B.listed_out.add(row)
                e += 1
                early = False
            else:
                if more:
                    fetch(r, row + 1)
                    fetched += 1
                B.listed_out.add(row)
                if r == 0:
                    loss[row] = "value"
            if more:
                B.listed.arrive()
            row += 1
            yield
        if sound:
            yield from leave(r, GW, row, sent, fetched)

    def computing(r, k):
        B = blocks[r]
        row = e = sent = 0
        early = False
        while row < rows and not early:
            if weights[row]:
                early = True
                if not (yield from wait(r, B.full, e)):
                    break
                need(B.buf == row or not sound, "a warp reads another row")
                yield
                need(B.buf == row or not sound, "overwritten while a warp reads it")
                if C > 1:
                    send_pairs(r, k, e, row)
                    sent = e + 1
                if not grad:
                    B.readers -= 1
                B.summed.arrive()
                yield
                if grad:
                    if not (yield from wait(r, *((B.xch[e % SETS], e // SETS) if C > 1 else (B.summed, e)))):
                        break
                    if C > 1:
                        got = B.pairs[e % SETS]
                        need(len(got) == GW * C and all(x == row for x in got.values()), "pairs of another row")
                    if not (yield from wait(r, B.listed, e)):
                        break
                    yield
                    need(B.buf == row or not sound, "overwritten while a warp reads it")
                    B.dense.setdefault(row, set()).add(k)
                    B.readers -= 1
                    B.empty.arrive()
                e += 1
                early = False
            else:
                B.dense.setdefault(row, set()).add(k)
            row += 1
            yield
        if sound:
            yield from leave(r, k, row, sent, 0)

    actors = [(r, computing(r, k)) for r in range(C) for k in range(GW)] + [(r, ahead(r)) for r in range(C)]
    weight = [rng.choice([0.05, 1.0, 1.0]) for _ in actors]
    landing = rng.choice([0.05, 0.5, 2.0])
    live = list(range(len(actors)))
    for _ in range(400000):
        if not live:
            break
        if flying and rng.random() < landing / (landing + 1):
            to, act = flying.pop(rng.randrange(len(flying)))
            need(blocks[to].gone < GW + 1, "a store lands in a block that has gone")
            act()
            continue
        i = rng.choices(live, weights=[weight[j] for j in live])[0]
        r, a = actors[i]
        try:
            next(a)
        except StopIteration:
            live.remove(i)
            blocks[r].gone += 1
            if blocks[r].gone == GW + 1:
                need(all(to != r for to, _ in flying), "a block goes with stores to it on their way")
    need(not live, "a warp never ends")
    for x in range(rows):
        need(loss[x] is not None, "a row without a loss")
        if loss[x] == "value":
            for B in blocks:
                need(x in B.listed_out, "a row that is not whole has a loss")
                need(not grad or len(B.dense.get(x, ())) == GW, "a row that is not whole has a loss")
    return loss.count("nan")


def batch(rng, n):
    kind = rng.random()
    if kind < 0.3:
        return [1] * n
    if kind < 0.4:
        return [0] * (n - 1) + [1]
    return [int(rng.random() < 0.7) for _ in range(n)]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("C", [1, 2, 4])
def test_every_wait_passes_when_none_runs_out(C, grad):
    rng = random.Random(C)
    for seed in range(60):
        assert run(C, grad, batch(rng, rng.randrange(1, 14)), seed, 0.0) == 0


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("C", [1, 2, 4])
def test_waits_that_run_out(C, grad):
    rng = random.Random(10 + C)
    marked = 0
    for seed in range(300):
        marked += run(C, grad, batch(rng, rng.randrange(1, 14)), seed, rng.choice([0.3, 0.02, 0.002, 0.0005])) > 0
    assert 30 < marked < 300      # both kinds of run are there


@pytest.mark.parametrize("grad", [False, True])
def test_going_on_after_a_wait_ran_out_is_a_fault(grad):
    rng = random.Random(5)
    faults = 0
    for seed in range(60):
        try:
            run(2, grad, batch(rng, 8), seed, 0.02, sound=False)
        except AssertionError:
            faults += 1
    assert faults > 20
