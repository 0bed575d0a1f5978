"""CPU model of the few-token layer's persistent launch.

Workgroups draw units of work -- route four tokens, 16 gate/up columns of an
expert, 32 output columns of an expert -- from one counter, in an order in
which a unit depends on units of lower numbers only.  Second-product units go
ahead once their expert's activations are there; the first one whose are not
waits for all of them: whoever drew the first of them watches the experts'
counters and tells every other workgroup on a word of its own.  Every wait is
bounded: one that takes too long is given up, and what a workgroup adds to the
result from then on is NaN.  A workgroup that gives up waiting for the routing
does no more and says so in a word that has the sum's launch (calls with routing
units have one) write NaN throughout.

The model replays that protocol (the scheduling wave's decisions, a queue of
descriptors, the draws held ahead) with random durations and workgroups that
start late, and checks what the kernel promises: with patience every output
block is right; without it every block is right or NaN, never a finite wrong
one, and the run ends.  It is a model of the protocol, not of the kernel's code.
"""
import random

import pytest

DESCS = 4
ROUTE, GATEUP, DOWN, EXIT = range(4)
CLAMP = 5


class Call:
    """One call: ``tokens`` (0: every workgroup routes them all itself), row
    blocks of each chosen expert, gate/up and output column blocks."""

    def __init__(self, tokens, blocks, per_g, per_d, nwg, seed, patience, late=0,
                 sleep_at=None):
        self.rnd = random.Random(seed)
        self.n_route, self.tokens = (tokens + 3) // 4, tokens
        self.blocks, self.per_g, self.per_d = blocks, per_g, per_d
        self.nwg, self.patience = nwg, patience
        self.now = self.asleep = 0           # (time in which nothing of the call ran)
        self.sleep_at = sleep_at
        self.next = self.routed = 0
        self.act = {}                        # finished gate/up units of an expert
        self.go = [0] * nwg                  # 1: the activations are complete, 2: given up
        self.unrouted = False
        self.per_col = sum(blocks)
        self.col_done = [0] * per_d
        self.yp = {}                         # (expert, row block, column): ok, wrong, nan
        self.y = [None] * per_d
        self.gus = [(e, rb, c) for e, nb in enumerate(blocks) for c in range(per_g)
                    for rb in range(nb)]
        self.downs = [(e, rb, c) for e, nb in enumerate(blocks) for c in range(per_d)
                      for rb in range(nb)]
        self.late = late

    def draw(self):
        self.next += 1
        return self.next - 1

    def complete(self, e):
        return self.act.get(e, 0) >= self.blocks[e] * self.per_g

    def waiter(self):
        """Asked after a look that found nothing: is the wait given up?  A step of
        the clock counts at most CLAMP, and a look follows the last of them."""
        last, spent, late = self.now + self.asleep, 0, False

        def give_up():
            nonlocal last, spent, late
            if late:
                return True
            now = self.now + self.asleep
            spent, last = spent + min(now - last, CLAMP), now
            late = spent >= self.patience
            return False
        return give_up

    def schedule(self, b, wg):
        """The scheduling wave of workgroup b; wg: queue, done, lost."""
        first_down = self.n_route + len(self.gus)
        held, held2 = self.draw(), None
        go = lost = False
        seq = 0
        while True:
            u = held
            while wg["done"] < seq - DESCS + 1:
                yield 1
            if u < self.n_route:
                unit = (ROUTE, u)
            else:
                if self.n_route and not wg.get("tables"):
                    give_up = self.waiter()
                    while self.routed < self.tokens and not lost:
                        lost = give_up()
                        yield 1
                    self.unrouted = self.unrouted or lost
                wg["tables"] = wg.get("tables") or not lost
                v = u - self.n_route
                if not wg["tables"]:
                    unit = (EXIT, None)
                elif v < len(self.gus):
                    unit = (GATEUP, self.gus[v])
                elif v < len(self.gus) + len(self.downs):
                    unit = (DOWN, self.downs[v - len(self.gus)])
                else:
                    unit = (EXIT, None)
            pending = False
            if unit[0] == DOWN and not go:
                word = self.go[b]
                there = word != 0 or self.complete(unit[1][0])
                go = word != 0
                lost = wg["lost"] = lost or word == 2
                pending = not there or u == first_down
            if not pending:
                wg["queue"].append(unit)
            if unit[0] == EXIT:
                return
            held = self.draw() if seq == 0 else held2
            held2 = self.draw()
            seq += 1
            if not pending:
                yield self.rnd.randint(1, 2)
                continue
            give_up = self.waiter()
            if u == first_down:
                while not all(self.complete(e) for e in range(len(self.blocks))) and not lost:
                    lost = give_up()
                    yield 1
                for w in range(self.nwg):
                    self.go[w] = 2 if lost else 1
            else:
                while self.go[b] == 0 and not lost:
                    lost = give_up()
                    yield 1
                lost = lost or self.go[b] == 2
            go = True
            wg["lost"] = wg["lost"] or lost
            wg["queue"].append(unit)

    def execute(self, b, wg):
        """The streaming and finishing waves of workgroup b."""
        seq = 0
        while True:
            while len(wg["queue"]) <= seq:
                yield 1
            kind, unit = wg["queue"][seq]
            if kind == EXIT:
                return
            if kind == DOWN:
                seen = self.complete(unit[0])
            yield self.rnd.randint(3, 40)
            if kind == ROUTE:
                self.routed += min(4, self.tokens - 4 * unit)
            elif kind == GATEUP:
                self.act[unit[0]] = self.act.get(unit[0], 0) + 1
            else:
                assert unit not in self.yp
                self.yp[unit] = "nan" if wg["lost"] else "ok" if seen else "wrong"
                c = unit[2]
                self.col_done[c] += 1
                if self.col_done[c] == self.per_col and not self.n_route:
                    self.sum(c)
            seq += 1
            wg["done"] = seq

    def sum(self, c):
        got = [self.yp.get((e, rb, c)) for e, nb in enumerate(self.blocks) for rb in range(nb)]
        self.y[c] = "nan" if "nan" in got else "wrong" if "wrong" in got or None in got else "ok"

    def run(self):
        gens, wake = {}, {}
        for b in range(self.nwg):
            wg = {"queue": [], "done": 0, "lost": False}
            t0 = self.rnd.choice([0, 0, 0, 60]) if self.late else 0
            for g in (self.schedule(b, wg), self.execute(b, wg)):
                gens[len(wake)] = g
                wake[len(wake)] = t0
        while gens:
            self.now += 1
            if self.now == self.sleep_at:
                self.asleep = 10 ** 9
            for i in list(gens):
                if wake[i] <= self.now:
                    try:
                        wake[i] = self.now + next(gens[i])
                    except StopIteration:
                        del gens[i]
            assert self.now < 10 ** 6, "the run does not end"
        if self.n_route:
            for c in range(self.per_d):
                self.sum(c)
                if self.unrouted:
                    self.y[c] = "nan"
        return self.y


SHAPES = [([1], 4, 2, 4), ([1, 1, 1], 8, 6, 16), ([1] * 7, 20, 12, 64), ([1, 2, 1], 6, 9, 8)]


@pytest.mark.parametrize("blocks,per_g,per_d,nwg", SHAPES)
@pytest.mark.parametrize("tokens", [0, 10, 61])
def test_with_patience_every_block_is_right(blocks, per_g, per_d, nwg, tokens):
    for seed in range(10):
        y = Call(tokens, blocks, per_g, per_d, nwg, seed, 10 ** 5, late=1).run()
        assert y == ["ok"] * per_d


@pytest.mark.parametrize("blocks,per_g,per_d,nwg", SHAPES)
@pytest.mark.parametrize("tokens", [0, 61])
def test_a_suspended_call_is_right(blocks, per_g, per_d, nwg, tokens):
    """The clock goes on while the GPU runs something else for long; the call's
    waits do not end by that."""
    for seed in range(4):
        for at in (2, 5, 20, 50, 100, 200):
            y = Call(tokens, blocks, per_g, per_d, nwg, seed, 10 ** 5, late=1, sleep_at=at).run()
            assert y == ["ok"] * per_d, (seed, at)


@pytest.mark.parametrize("blocks,per_g,per_d,nwg", SHAPES)
def test_a_watch_given_up_ends_in_nan(blocks, per_g, per_d, nwg):
    """Whoever gives up watching tells the others so, not that all is there."""
    seen = set()
    for seed in range(10):
        for patience in (0, 5, 20):
            y = Call(0, blocks, per_g, per_d, nwg, seed, patience, late=1).run()
            assert set(y) <= {"ok", "nan"}, (seed, patience, y)
            seen |= set(y)
    assert "nan" in seen


@pytest.mark.parametrize("tokens", [9, 61, 128])
@pytest.mark.parametrize("blocks,per_g,per_d,nwg", SHAPES)
def test_a_wait_for_the_routing_given_up_ends_in_nan(blocks, per_g, per_d, nwg, tokens):
    seen = set()
    for seed in range(10):
        for patience in (0, 5, 20, 60):
            y = Call(tokens, blocks, per_g, per_d, nwg, seed, patience, late=1).run()
            assert set(y) <= {"ok", "nan"}, (seed, patience, y)
            seen |= set(y)
    assert "nan" in seen


@pytest.mark.parametrize("impatient", [1, 2, 5])
def test_one_workgroup_that_gives_up_the_routing(impatient):
    """It alone: the others find its units missing, and give up in turn."""
    for seed in range(20):
        c = Call(61, [1, 1, 1], 8, 6, 16, seed, 3000)
        waiter, asked = c.waiter, iter(range(1000))
        c.waiter = lambda: (lambda: True) if next(asked) == impatient else waiter()
        assert set(c.run()) <= {"ok", "nan"}
