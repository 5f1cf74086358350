"""A small simulator for the barrier protocols of the tensor-core kernels: the
roles of one CTA as generators over mbarriers, named barriers and memory cells.

What it knows:
  - an mbarrier phase completes with its last arrival, and a wait may give up
    (as the kernels' limited waits do, each on its own): a random one of them
    when nobody can go on, and with probability `rush` one whose phase is only
    late;
  - a named barrier has no limit, and counts only threads that name the same
    number of them;
  - memory accesses are ordered only by what the barriers order (vector
    clocks), so a conflict is found in every schedule, not only in the one that
    loses; the tensor pipe runs in the order of its issue, behind its lane.

Roles yield tuples: ("wait", bar, parity) -> did it complete; ("arrive", bar);
("named", id, threads, value) -> the values or-ed; ("read"/"write", cell);
("mma", reads, writes) on the tensor pipe; ("commit", bar) behind all of it."""
import random


class Race(AssertionError):
    pass


class Hang(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0
        self.clock, self.seen = {}, {}

    def arrive(self, clock):
        join(self.clock, clock)
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1
            self.seen, self.clock = self.clock, {}

    def over(self, parity):  # the phase of this parity
        return (self.done & 1) != parity


def join(a, b):
    for k, v in b.items():
        if v > a.get(k, 0):
            a[k] = v


class Sim:
    def __init__(self, bars, seed=0, rush=0.0):
        self.bars = {k: Bar(n) for k, n in bars.items()}
        self.rng, self.rush = random.Random(seed), rush
        self.roles, self.clock, self.op, self.answer = {}, {}, {}, {}
        self.named = {}
        self.cells = {}
        self.gave_up = []

    def add(self, name, role):
        self.roles[name], self.clock[name] = role, {name: 1}
        self.answer[name] = None
        self._next(name)

    def _next(self, name):
        try:
            self.op[name] = self.roles[name].send(self.answer[name])
            self.answer[name] = None
        except StopIteration:
            self.op[name] = None

    def _access(self, who, clock, cell, write):
        if self.gave_up:  # after that nothing is ordered any more
            return
        last, reads = self.cells.setdefault(cell, [None, []])
        against = ([last] if last else []) + (reads if write else [])
        for other, at in against:
            if clock.get(other, 0) < at:
                raise Race(f"{who} {'writes' if write else 'reads'} {cell} beside {other}")
        if write:
            self.cells[cell] = [(who, clock[who]), []]
        else:
            reads.append((who, clock[who]))

    def _step(self, name):
        """Runs the role's operation if it can; False: it has to wait."""
        op, clock = self.op[name], self.clock[name]
        if op[0] == "wait":
            bar = self.bars[op[1]]
            if not bar.over(op[2]):
                return False
            join(clock, bar.seen)
            self.answer[name] = True
        elif op[0] == "arrive":
            self.bars[op[1]].arrive(clock)
        elif op[0] in ("read", "write"):
            self._access(name, clock, op[1], op[0] == "write")
        elif op[0] in ("mma", "commit"):
            pipe = self.clock.setdefault("pipe", {"pipe": 1})
            if op[0] == "mma":
                join(pipe, clock)
                for c in op[1]:
                    self._access("pipe", pipe, c, False)
                for c in op[2]:
                    self._access("pipe", pipe, c, True)
            else:
                self.bars[op[1]].arrive(pipe)
            pipe["pipe"] += 1
        else:
            _, bar, threads, value = op
            there = self.named.setdefault(bar, {})
            if name not in there:
                if any(t != threads for t, _ in there.values()):
                    raise Hang(f"barrier {bar}: {name} names {threads} threads, others another number")
                there[name] = (threads, value)
            if len(there) * 32 < threads:
                return False
            both = {}
            for n in there:
                join(both, self.clock[n])
            result = any(v for _, v in there.values())
            self.named[bar] = {}
            for n in there:
                join(self.clock[n], both)
                self.clock[n][n] += 1
                self.answer[n] = result
                self._next(n)
            return True
        clock[name] += 1
        self._next(name)
        return True

    def _give_up(self, name):
        self.gave_up.append((name, self.op[name][1]))
        self.answer[name] = False
        self.clock[name][name] += 1
        self._next(name)

    def run(self):
        while True:
            alive = [n for n in self.roles if self.op[n] is not None]
            if not alive:
                return
            self.rng.shuffle(alive)
            stuck = [n for n in alive if self.op[n][0] == "wait" and not self.bars[self.op[n][1]].over(self.op[n][2])]
            if stuck and self.rng.random() < self.rush:
                self._give_up(stuck[0])
            elif not any(self._step(n) for n in alive):
                if not stuck:
                    raise Hang("for ever at " + ", ".join(f"{n}: {self.op[n][1]}" for n in alive))
                self._give_up(stuck[0])


class Waiter:
    """mbar_wait of one thread (or warp): after one that ran out, none waits."""

    def __init__(self):
        self.failed = False

    def wait(self, bar, parity):
        if self.failed:
            return False
        if not (yield ("wait", bar, parity & 1)):
            self.failed = True
        return not self.failed
