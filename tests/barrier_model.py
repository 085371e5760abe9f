"""A host model of the barriers of the warp-specialised cross-attention kernels.

A kernel is a set of agents (its warps, each a generator of operations) that share mbarriers and
buffers. A barrier completes a phase when its count of arrivals is in; a wait for phase p looks at
the parity of the completed phases only, as the hardware does. So it is sound only while phase p - 1
has completed and phase p + 1 has not: a wait that could pass before its phase, or be overtaken by
the next one, raises Violation, as does a buffer that is read while it does not hold what the reader
expects, or written while somebody reads it, and a state in which nothing can move.

Copies complete in any order, an agent's products in the order in which it issued them. Schedules
are random, or starve one agent, one queue of products or one kind of copy: it moves only when
nothing else can.
"""
import random


class Violation(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.completed = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.completed = self.count, self.completed + 1

    def test(self, phase):
        return (self.completed - 1 - phase) % 2 == 0


class Buf:
    """What a buffer holds; its readers and writers still under way."""

    def __init__(self):
        self.holds, self.readers, self.writers, self.owner = None, 0, 0, None


class Machine:
    def __init__(self):
        self.bars, self.bufs, self.agents, self.queues, self.copies = {}, {}, [], {}, []
        self.trace = []

    # ---- set up
    def bar(self, name, count=1):
        self.bars[name] = Bar(count)

    def agent(self, name, gen):
        self.agents.append([name, gen, None])
        self.queues[name] = []

    # ---- buffers
    def buf(self, name):
        return self.bufs.setdefault(name, Buf())

    def reads(self, name, tag, who):
        b = self.buf(name)
        if b.writers or b.holds != tag:
            raise Violation(f"{who} reads {name}: holds {b.holds}{' (being written)' if b.writers else ''}, "
                            f"expects {tag}")

    def writes(self, name, who, adds=False):
        """adds: a product onto the sums of the same agent's earlier ones, which complete in order."""
        b = self.buf(name)
        if b.readers or (b.writers and not (adds and b.owner == who)):
            raise Violation(f"{who} writes {name} ({b.holds}) while it is read or written")

    # ---- operations of an agent: (kind, ...)
    #   wait bar phase | probe bar phase | arrive bar | read buf tag | write buf tag
    #   products [(buf, tag) read] [(buf, tag, adds) written] [bars committed]   in order, per agent
    #   copy kind buf tag bar                                      complete in any order
    #   store buf tag: a copy out of buf, and the wait for its end
    def enabled(self, a):
        op = a[2]
        return op[0] != "wait" or self.bars[op[1]].test(op[2])

    def advance(self, a, value=None):
        try:
            a[2] = a[1].send(value)
        except StopIteration:
            a[2] = None
            return
        if a[2][0] == "wait":
            self.look(a)

    def look(self, a):
        _, bar, phase = a[2][:3]
        b = self.bars[bar]
        if b.completed > phase + 1:
            raise Violation(f"{a[0]} waits for phase {phase} of {bar}: overtaken, {b.completed} are complete")

    def step(self, a):
        op, who, value = a[2], a[0], None
        kind = op[0]
        if kind in ("wait", "probe"):
            b = self.bars[op[1]]
            value = b.test(op[2])
            if value and b.completed < op[2] + 1 and op[2] >= 0:
                raise Violation(f"{who} passes phase {op[2]} of {op[1]}: {b.completed} are complete")
        elif kind == "arrive":
            self.arrive(op[1])
        elif kind == "read":
            self.reads(op[1], op[2], who)
        elif kind == "write":
            self.writes(op[1], who)
            self.buf(op[1]).holds = op[2]
        elif kind == "products":
            _, ins, outs, bars = op
            for name, tag in ins:
                self.reads(name, tag, who)
                self.buf(name).readers += 1
            for name, _, adds in outs:
                self.writes(name, who, adds)
                b = self.buf(name)
                b.writers += 1
                b.owner = who
            self.queues[who].append((ins, outs, bars))
        elif kind == "copy":
            _, label, buf, tag, bar = op
            self.writes(buf, who)
            self.buf(buf).writers += 1
            self.copies.append((label, buf, tag, bar))
        elif kind == "store":
            self.reads(op[1], op[2], who)
            self.buf(op[1]).readers += 1
            self.copies.append(("store", op[1], None, a))
            a[2] = ("stored",)
            return
        elif kind == "stored":
            return
        self.advance(a, value)

    def arrive(self, bar):
        b = self.bars[bar]
        before = b.completed
        b.arrive()
        if b.completed != before:
            for a in self.agents:
                if a[2] is not None and a[2][0] == "wait" and a[2][1] == bar:
                    self.look(a)

    def finish_products(self, who):
        ins, outs, bars = self.queues[who].pop(0)
        for name, tag in ins:
            b = self.buf(name)
            b.readers -= 1
            if b.holds != tag:
                raise Violation(f"{name} changed from {tag} to {b.holds} under a product of {who}")
        for name, tag, _ in outs:
            b = self.buf(name)
            b.writers -= 1
            b.holds = tag
        for bar in bars:
            self.arrive(bar)

    def finish_copy(self, i):
        label, buf, tag, bar = self.copies.pop(i)
        b = self.buf(buf)
        if label == "store":
            b.readers -= 1
            self.advance(bar)
            return
        b.writers -= 1
        b.holds = tag
        self.arrive(bar)

    # ---- a run under a schedule
    def run(self, rng, starved=None):
        for a in self.agents:
            self.advance(a)
        while True:
            acts = [("agent", a[0], a) for a in self.agents
                    if a[2] is not None and a[2][0] != "stored" and self.enabled(a)]
            acts += [("products", who, who) for who, q in self.queues.items() if q]
            acts += [("copy", c[0], i) for i, c in enumerate(self.copies)]
            if not acts:
                left = [(a[0], a[2]) for a in self.agents if a[2] is not None]
                if left:
                    raise Violation(f"nothing can move: {left}")
                return
            if starved is not None:
                fed = [x for x in acts if x[:2] != starved]
                acts = fed or acts
            kind, _, key = rng.choice(acts)
            if kind == "agent":
                self.step(key)
            elif kind == "products":
                self.finish_products(key)
            else:
                self.finish_copy(key)

    def parties(self):
        """What a schedule can starve."""
        return [("agent", a[0]) for a in self.agents] + [("products", a[0]) for a in self.agents] + \
            [("copy", x) for x in ("K", "V", "Q", "G", "R", "KV", "store")]


def check(build, seeds=1):
    """Runs the kernel that build() returns under random schedules and starving each party."""
    for starved in [None] + build().parties():
        for seed in range(seeds if starved else 6 * seeds):
            m = build()
            try:
                m.run(random.Random(seed), starved)
            except Violation as e:
                raise Violation(f"{e} (starved: {starved}, seed {seed})") from None


# ------------------------------------------------------------------ k_cross_dkv
def dkv(c, steps):
    """c: stages, five (slots of S, dP, P and dS), turns: barriers that P full and products done of
    consecutive steps take turns on."""
    m = Machine()
    NS, five, NT = c["stages"], c["five"], c["turns"]
    m.bar("AFULL")
    m.bar("ALL")
    for i in range(NS):
        m.bar(("QFULL", i))
        m.bar(("QEMPTY", i))
    for i in range(2):
        m.bar(("SFULL", i))
        m.bar(("SFREE", i), 4)
    for i in range(NT):
        m.bar(("PFULL", i), 4)
        m.bar(("DONE", i))
    s = (lambda i: i % 5) if five else (lambda i: 2 * (i & 1))
    g = (lambda i: s(i + 2)) if five else (lambda i: s(i) + 1)

    def elementwise(b, w):
        seen = False
        for i in range(b, steps, 2):
            if not seen:
                yield "wait", ("SFULL", b), i >> 1
            yield "wait", ("QFULL", i % NS), i // NS
            yield "read", ("rows", i % NS), i
            yield "read", ("T", s(i), w), ("S", i)
            yield "read", ("T", g(i), w), ("dP", i)
            if five:
                yield "arrive", ("SFREE", b)
            yield "write", ("T", s(i), w), ("P", i)
            seen = (yield "probe", ("SFULL", b), (i >> 1) + 1) if five else False
            yield "arrive", ("PFULL", i % NT)
        yield "wait", "ALL", 0
        yield "read", ("dkv",), steps - 1

    def loads():
        yield "copy", "K", ("KV",), 0, "AFULL"
        for i in range(steps):
            st = i % NS
            if i >= NS:
                yield "wait", ("QEMPTY", st), i // NS - 1
            yield "copy", "Q", ("rows", st), i, ("QFULL", st)

    def scores():
        yield "wait", "AFULL", 0
        for i in range(steps):
            yield "wait", ("QFULL", i % NS), i // NS
            done = i - (3 if five else 2)
            if five and i >= 2:
                yield "wait", ("SFREE", i & 1), (i - 2) >> 1
            if done >= 0:
                yield "wait", ("DONE", done % NT), done // NT
            yield "products", [(("rows", i % NS), i), (("KV",), 0)], \
                [(("T", s(i), w), ("S", i), 0) for w in range(4)] + \
                [(("T", g(i), w), ("dP", i), 0) for w in range(4)], [("SFULL", i & 1)]

    def product():
        for i in range(steps):
            yield "wait", ("PFULL", i % NT), i // NT
            yield "products", [(("T", s(i), w), ("P", i)) for w in range(4)] + [(("rows", i % NS), i)], [], \
                [("QEMPTY", i % NS)]
            yield "products", [], [(("dkv",), i, 1)], [("DONE", i % NT)] + (["ALL"] if i + 1 == steps else [])

    for b in range(2):
        for w in range(4):
            m.agent(f"elementwise {b}.{w}", elementwise(b, w))
    m.agent("loads", loads())
    m.agent("S products", scores())
    m.agent("dk, dv products", product())
    return m
