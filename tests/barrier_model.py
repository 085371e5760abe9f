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


# ------------------------------------------------------------------ k_cross_fwd
def forward(c, units, masked):
    """units: [(row tiles, state tiles)] of one CTA. c: slots, bufs, ready."""
    m = Machine()
    NS, NB, NR = c["slots"], c["bufs"], c["ready"]
    for i in range(NS):
        m.bar(("FULL", i))
        m.bar(("EMPTY", i), 2)
    for i in range(NR):
        m.bar(("READY", i))
    for t in range(2):
        for b in range(2):
            m.bar(("QFULL", b, t))
            m.bar(("QEMPTY", b, t))
            m.bar(("SFULL", b, t))
            m.bar(("SFREE", b, t), 4)
            m.bar(("SUM", b, t), 4)
        for n, k in (("PFULL", 4), ("DONE", 1), ("OFULL", 1), ("OFREE", 4), ("STAGED", 4)):
            m.bar((n, t), k)

    def softmax(t, w):
        gc = uc = 0
        for nt, nj in units:
            if (t == 1 and nt < 2) or not nj:
                continue
            seen = False
            for j in range(nj):
                b = gc % NB
                if not seen:
                    yield "wait", ("SFULL", b, t), gc // NB
                yield "read", ("S", t, b), gc
                yield "arrive", ("SFREE", b, t)
                if gc % 3 == 2 and j:  # O is rescaled
                    yield "wait", ("DONE", t), gc - 1
                    yield "read", ("O", t), (uc, j - 1)
                done = yield "probe", ("DONE", t), gc - 1
                seen = yield "probe", ("SFULL", (gc + 1) % NB, t), (gc + 1) // NB
                if gc and not done:
                    yield "wait", ("DONE", t), gc - 1
                yield "write", ("P", t, w), gc
                if j + 1 == nj:
                    yield "write", ("sum", uc & 1, t, w), uc
                    yield "arrive", ("SUM", uc & 1, t)
                yield "arrive", ("PFULL", t)
                gc += 1
            uc += 1

    def epilogue(w):
        uc = [0, 0]
        for nt, nj in units:
            if not nj:
                continue
            for t in range(nt):
                turn = uc[t] & 1
                yield "wait", ("SUM", turn, t), uc[t] >> 1
                yield "wait", ("OFULL", t), uc[t]
                yield "read", ("sum", turn, t, w), uc[t]
                yield "read", ("O", t), (uc[t], nj - 1)
                yield "write", ("Q", turn, t, w), ("out", uc[t])
                yield "arrive", ("STAGED", t)
                yield "arrive", ("OFREE", t)
                if w == 0:
                    yield "wait", ("STAGED", t), uc[t]
                    for x in range(4):
                        yield "store", ("Q", turn, t, x), ("out", uc[t])
                    yield "arrive", ("QEMPTY", turn, t)
                uc[t] += 1

    def loads():
        kv, uc = 0, [0, 0]
        for nt, nj in units:
            if not nj:
                continue
            for t in range(nt):
                n = uc[t]
                if n >= 2:
                    yield "wait", ("QEMPTY", n & 1, t), (n >> 1) - 1
                for x in range(3):  # the quarters of the tile land together: the last one's copy arrives
                    yield "write", ("Q", n & 1, t, x), n
                yield "copy", "Q", ("Q", n & 1, t, 3), n, ("QFULL", n & 1, t)
                uc[t] += 1
            for j in range(2 * nj):
                st = kv % NS
                if kv >= NS:
                    yield "wait", ("EMPTY", st), kv // NS - 1
                yield "copy", "KV"[j & 1], ("ring", st), kv, ("FULL", st)
                kv += 1

    def scores(t):
        kv = n = uc = 0
        for nt, nj in units:
            if not nj:
                continue
            mine = t < nt
            if mine:
                yield "wait", ("QFULL", uc & 1, t), uc >> 1
            for _ in range(nj):
                st, b = 2 * kv % NS, n % NB
                wait = mine and n >= NB
                pf = yield "probe", ("FULL", st), 2 * kv // NS
                pe = (yield "probe", ("SFREE", b, t), n // NB - 1) if wait else True
                if not pf:
                    yield "wait", ("FULL", st), 2 * kv // NS
                if not pe:
                    yield "wait", ("SFREE", b, t), n // NB - 1
                if mine:
                    q = [(("Q", uc & 1, t, x), uc) for x in range(4)]
                    yield "products", q + [(("ring", st), 2 * kv)], [(("S", t, b), n, 0)], [("SFULL", b, t)]
                yield "products", [], [], [("EMPTY", st)]
                n += mine
                kv += 1
            uc += mine

    def outputs(t):
        kv = n = uc = 0
        for nt, nj in units:
            if not nj:
                continue
            mine = t < nt
            if mine and uc:
                yield "wait", ("OFREE", t), uc - 1
            for j in range(nj):
                st = (2 * kv + 1) % NS
                vb = ("READY", kv % NR) if masked else ("FULL", st)
                vp = kv // NR if masked else (2 * kv + 1) // NS
                pv = yield "probe", vb, vp
                if mine:
                    yield "wait", ("PFULL", t), n
                if not pv:
                    yield "wait", vb, vp
                if mine:
                    ins = [(("P", t, w), n) for w in range(4)] + [(("ring", st), ("cleared", 2 * kv + 1)
                                                                   if masked else 2 * kv + 1)]
                    yield "products", ins, [(("O", t), (uc, j), 1)], [("DONE", t)]
                    if j + 1 == nj:
                        yield "products", [], [], [("OFULL", t)]
                yield "products", [], [], [("EMPTY", st)]
                n += mine
                kv += 1
            uc += mine

    def clear():
        g = 0
        for _, nj in units:
            for _ in range(nj):
                kv = 2 * g + 1
                yield "wait", ("FULL", kv % NS), kv // NS
                yield "read", ("ring", kv % NS), kv
                yield "write", ("ring", kv % NS), ("cleared", kv)
                yield "arrive", ("READY", g % NR)
                g += 1

    for t in range(2):
        for w in range(4):
            m.agent(f"softmax {t}.{w}", softmax(t, w))
        m.agent(f"S products {t}", scores(t))
        m.agent(f"O products {t}", outputs(t))
    for w in range(4):
        m.agent(f"epilogue {w}", epilogue(w))
    m.agent("loads", loads())
    if masked:
        m.agent("clear", clear())
    return m


# ------------------------------------------------------------------ k_cross_dq
def dq(c, units, masked):
    """units: steps of 64 states of each unit. c: slots, ready, own (dS has columns of its own)."""
    m = Machine()
    NS, NR, own = c["slots"], c["ready"], c["own"]
    for n, k in (("QFULL", 1), ("QEMPTY", 1), ("SFULL", 1), ("SFREE", 4), ("PFULL", 4), ("DONE", 1),
                 ("STAGED", 4)):
        m.bar(n, k)
    for i in range(NS):
        m.bar(("FULL", i))
        m.bar(("EMPTY", i))
    for i in range(NR):
        m.bar(("READY", i))
    dS = (lambda w: ("dS", w)) if own else (lambda w: ("S", w))

    def elementwise(w):
        gc = uc = 0
        for n in units:
            if not n:
                continue
            yield "wait", "QFULL", uc
            yield "read", ("G",), uc
            seen = False
            for j in range(n):
                if not seen:
                    yield "wait", "SFULL", gc
                done = yield "probe", "DONE", gc - 1
                yield "read", ("S", w), ("S", gc)
                yield "read", ("dP",), gc
                if own:
                    yield "arrive", "SFREE"
                    if gc and not done:
                        yield "wait", "DONE", gc - 1
                yield "write", dS(w), ("dS", gc)
                seen = (yield "probe", "SFULL", gc + 1) if own else False
                yield "arrive", "PFULL"
                gc += 1
            yield "wait", "DONE", gc - 1
            yield "read", ("dq",), (uc, n - 1)
            yield "write", ("Q", w), ("out", uc)
            yield "arrive", "STAGED"
            if w == 0:
                yield "wait", "STAGED", uc
                for x in range(4):
                    yield "store", ("Q", x), ("out", uc)
                yield "arrive", "QEMPTY"
            uc += 1

    def loads():
        kv = uc = 0
        for n in units:
            if not n:
                continue
            if uc:
                yield "wait", "QEMPTY", uc - 1
            for x in range(4):
                yield "write", ("Q", x), uc
            yield "copy", "Q", ("G",), uc, "QFULL"
            uc += 1
            for _ in range(n):
                for x in range(2):
                    st = kv % NS
                    if kv >= NS:
                        yield "wait", ("EMPTY", st), kv // NS - 1
                    yield "copy", "VK"[x], ("ring", st), kv, ("FULL", st)
                    kv += 1

    def scores():
        g = uc = 0
        for n in units:
            if not n:
                continue
            yield "wait", "QFULL", uc
            for _ in range(n):
                sv, sk = 2 * g % NS, (2 * g + 1) % NS
                if masked:
                    yield "wait", ("READY", g % NR), g // NR
                else:
                    yield "wait", ("FULL", sk), (2 * g + 1) // NS
                yield "wait", ("FULL", sv), 2 * g // NS
                if g:
                    yield "wait", "SFREE" if own else "DONE", g - 1
                k = ("cleared", 2 * g + 1) if masked else 2 * g + 1
                yield "products", [(("Q", x), uc) for x in range(4)] + [
                    (("G",), uc), (("ring", sk), k), (("ring", sv), 2 * g)], \
                    [(("S", w), ("S", g), 0) for w in range(4)] + [(("dP",), g, 0)], ["SFULL", ("EMPTY", sv)]
                g += 1
            uc += 1

    def product():
        g = 0
        for u, n in enumerate(x for x in units if x):
            for j in range(n):
                sk = (2 * g + 1) % NS
                yield "wait", "PFULL", g
                k = ("cleared", 2 * g + 1) if masked else 2 * g + 1
                yield "products", [(dS(w), ("dS", g)) for w in range(4)] + [(("ring", sk), k)], \
                    [(("dq",), (u, j), 1)], ["DONE", ("EMPTY", sk)]
                g += 1

    def clear():
        g = 0
        for n in units:
            for _ in range(n):
                kv = 2 * g + 1
                yield "wait", ("FULL", (kv - 1) % NS), (kv - 1) // NS
                yield "wait", ("FULL", kv % NS), kv // NS
                yield "read", ("ring", kv % NS), kv
                yield "write", ("ring", kv % NS), ("cleared", kv)
                yield "arrive", ("READY", g % NR)
                g += 1

    for w in range(4):
        m.agent(f"elementwise {w}", elementwise(w))
    m.agent("loads", loads())
    m.agent("S products", scores())
    m.agent("dq products", product())
    if masked:
        m.agent("clear", clear())
    return m


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


# ------------------------------------------------------------------ k_cross_fwd_short
def forward_short(c, run):
    """run: row tiles of each problem that the CTA walks. c: staged (barriers of staged rows)."""
    m = Machine()
    NG = c["staged"]
    units = [(p, i) for p, n in enumerate(run) for i in range(n)]
    for n, k in (("KV", 1), ("VREADY", 4), ("S", 1), ("P", 4), ("O", 1)):
        m.bar(n, k)
    for i in range(2):
        m.bar(("Q", i))
        m.bar(("QFREE", i))
    for i in range(NG):
        m.bar(("STAGED", i), 4)

    def softmax(w):
        for n, (p, i) in enumerate(units):
            if i == 0:
                yield "wait", "KV", p
                yield "read", ("KV", w), p
                yield "write", ("KV", w), ("cleared", p)
                yield "arrive", "VREADY"
            yield "wait", "S", n
            yield "read", ("S", w), ("S", n)
            yield "write", ("S", w), ("P", n)
            yield "arrive", "P"
            yield "wait", "O", n
            yield "read", ("O",), n
            yield "write", ("Q", n & 1, w), ("out", n)
            yield "arrive", ("STAGED", n % NG)

    def products():
        gen = 0

        def load(i):
            for x in range(3):
                yield "write", ("Q", i & 1, x), i
            yield "copy", "Q", ("Q", i & 1, 3), i, ("Q", i & 1)

        yield from load(0)
        for n, (p, i) in enumerate(units):
            if n:
                yield "wait", "O", n - 1
            if i == 0:
                for x in range(3):
                    yield "write", ("KV", x), p
                yield "copy", "KV", ("KV", 3), p, "KV"
                yield "wait", "KV", gen
                gen += 1
            yield "wait", ("Q", n & 1), n >> 1
            yield "products", [(("Q", n & 1, x), n) for x in range(4)], [(("S", w), ("S", n), 0) for w in range(4)], \
                ["S"]
            if n + 1 < len(units):
                if n >= 1:
                    yield "wait", ("QFREE", (n + 1) & 1), ((n + 1) >> 1) - 1
                yield from load(n + 1)
            if i == 0:
                yield "wait", "VREADY", gen - 1
            yield "wait", "P", n
            yield "products", [(("S", w), ("P", n)) for w in range(4)] + \
                [(("KV", w), ("cleared", p)) for w in range(4)], [(("O",), n, 0)], ["O"]

    def stores():
        for n in range(len(units)):
            yield "wait", ("STAGED", n % NG), n // NG
            for x in range(4):
                yield "store", ("Q", n & 1, x), ("out", n)
            yield "arrive", ("QFREE", n & 1)

    for w in range(4):
        m.agent(f"softmax {w}", softmax(w))
    m.agent("products", products())
    m.agent("stores", stores())
    return m


# ------------------------------------------------------------------ k_cross_bwd_short
def backward_short(c, run):
    """run: row tiles of each problem that the CTA walks. c: bufs (buffers of P and dS)."""
    m = Machine()
    bufs = c["bufs"]
    units = [(p, i, i + 1 == n) for p, n in enumerate(run) for i in range(n)]
    N = len(units)
    for n, k in (("KV", 1), ("KREADY", 4), ("S", 1), ("SFREE", 4), ("DQFREE", 4), ("FLUSH", 4), ("STAGED", 4),
                 ("STFREE", 1)):
        m.bar(n, k)
    for i in range(2):
        for n, k in (("Q", 1), ("ROWS", 4), ("PD", 4), ("MM", 1)):
            m.bar((n, i), k)

    def elementwise(w):
        for n, (p, i, _) in enumerate(units):
            if i == 0:
                yield "wait", "KV", p
                yield "read", ("KV", w), p
                yield "write", ("KV", w), ("cleared", p)
                yield "arrive", "KREADY"
            yield "wait", ("ROWS", n & 1), n >> 1
            yield "wait", "S", n
            if n >= bufs:
                yield "wait", ("MM", (n - bufs) & 1), (n - bufs) >> 1
            yield "read", ("srow", n & 1, w), n
            yield "read", ("S",), n
            yield "arrive", "SFREE"
            yield "write", ("PD", n % bufs, w), n
            yield "arrive", ("PD", n & 1)

    def rows(w):
        def of(i):
            yield "wait", ("Q", i & 1), i >> 1
            yield "read", ("Q", i & 1), i
            yield "write", ("srow", i & 1, w), i
            yield "arrive", ("ROWS", i & 1)

        yield from of(0)
        for n, (p, i, last) in enumerate(units):
            if n + 1 < N:
                yield from of(n + 1)
            yield "wait", ("MM", n & 1), n >> 1
            if n:
                yield "wait", "STFREE", n - 1
            yield "read", ("dq",), n
            yield "write", ("out", w), n
            yield "arrive", "STAGED"
            yield "arrive", "DQFREE"
            if last:
                yield "read", ("dkv",), (p, i)
                yield "arrive", "FLUSH"

    def moves():
        loaded = 0
        while loaded < min(2, N):
            yield "copy", "Q", ("Q", loaded & 1), loaded, ("Q", loaded & 1)
            loaded += 1
        for n in range(N):
            if loaded < N:
                yield "wait", ("MM", n & 1), n >> 1
                yield "copy", "Q", ("Q", loaded & 1), loaded, ("Q", loaded & 1)
                loaded += 1
            yield "wait", "STAGED", n
            for x in range(4):
                yield "store", ("out", x), n
            yield "arrive", "STFREE"

    def products():
        gen = issued = 0

        def scores(i):
            p = units[i][0]
            yield "products", [(("Q", i & 1), i)] + [(("KV", w), ("cleared", p)) for w in range(4)], \
                [(("S",), i, 0)], ["S"]

        for n, (p, i, _) in enumerate(units):
            if issued == n:
                if i == 0:
                    if n:
                        yield "wait", ("MM", (n - 1) & 1), (n - 1) >> 1
                        yield "wait", "FLUSH", gen - 1
                    for x in range(3):
                        yield "write", ("KV", x), p
                    yield "copy", "KV", ("KV", 3), p, "KV"
                    gen += 1
                    yield "wait", "KV", gen - 1
                    yield "wait", "KREADY", gen - 1
                yield "wait", ("Q", n & 1), n >> 1
                if n:
                    yield "wait", "SFREE", n - 1
                yield from scores(n)
                issued += 1
            yield "wait", "SFREE", n
            if n + 1 < N and units[n + 1][1] != 0:
                there = yield "probe", ("Q", (n + 1) & 1), (n + 1) >> 1
                if there:
                    yield from scores(n + 1)
                    issued += 1
            yield "wait", ("PD", n & 1), n >> 1
            if n:
                yield "wait", "DQFREE", n - 1
            yield "products", [(("PD", n % bufs, w), n) for w in range(4)] + [(("Q", n & 1), n)] + \
                [(("KV", w), ("cleared", p)) for w in range(4)], [(("dq",), n, 0), (("dkv",), (p, i), 1)], \
                [("MM", n & 1)]

    for w in range(4):
        m.agent(f"elementwise {w}", elementwise(w))
    for w in range(4):
        m.agent(f"rows {w}", rows(w))
    m.agent("moves", moves())
    m.agent("products", products())
    return m
