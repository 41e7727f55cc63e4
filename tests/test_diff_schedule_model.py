"""Models of the barrier protocols of the three differential attention kernels
(csrc/diff_fwd.cu, diff_dq_kernel and diff_dkv_kernel of csrc/diff_bwd.cu), checked on CPU
for deadlock and stale data over randomised interleavings.

The agents are the kernels' roles: loading warps, MMA-issuing threads, eight elementwise
warps.  TMA loads complete in any order.  The MMAs of one issuing thread execute in issue
order, those of two threads in any order between them; a commit arrives once every MMA its
own thread issued before has executed.  An mbarrier wait on parity p succeeds once the phase
with parity p has completed, as try_wait.parity does.  An agent can be interrupted between a
wait and what follows it, and between a read and the arrival that reports it.

Every buffer (a stage of a ring, an item's fixed operands, columns of tensor memory, the row
sums' exchange) knows the version it holds, the parts of it that are written and who has still
to read it.  A read checks version and completeness; a write checks that the version before has been
read by all its readers.  Planted ordering mistakes show that the checks catch what they should.
"""
import random

import pytest

WARPS = range(8)


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return (self.phase & 1) != parity


class Buf:
    """Versions with parts and readers.  need(version): names of the reads it must see before a write."""

    def __init__(self, name, need, parts=1):
        self.name, self.need, self.parts = name, need, parts
        self.version, self.have, self.left = None, 0, set()

    def write(self, version):
        """One part of ``version``; the first part starts it."""
        if version != self.version:
            assert not self.left, f"{self.name}: {version} written over {self.version}, unread by {sorted(map(str, self.left))}"
            assert self.version is None or self.have == self.parts, f"{self.name}: {version} over an incomplete {self.version}"
            self.version, self.have, self.left = version, 0, set(self.need(version))
        self.have += 1
        assert self.have <= self.parts

    def read(self, version, who):
        assert self.version == version and self.have == self.parts, \
            f"{self.name}: {who} wants {version}, finds {self.version} ({self.have} of {self.parts} parts)"
        self.left.discard(who)


class Model:
    def __init__(self, items, seed, mutation):
        self.rng, self.items, self.mutation = random.Random(seed), items, mutation
        self.blocks = [(k, j) for k, n in enumerate(items) for j in range(n)]
        self.first = [sum(items[:k]) for k in range(len(items))]
        self.bars, self.bufs = {}, {}
        self.mma = {}        # issuing thread: queue of functions
        self.commits = {}    # issuing thread: (MMAs issued before, barrier)
        self.count = {}      # issuing thread: issued, executed
        self.loads = []

    def bar(self, name, count=1, n=None):
        for i in ([""] if n is None else range(n)):
            self.bars[f"{name}{i}"] = Bar(count)

    def buf(self, name, need, parts=1):
        self.bufs[name] = Buf(name, need, parts)

    # ------------------------------------------------------------ asynchronous units
    def load(self, buf, version, bar):
        b = self.bufs[buf]
        assert not b.left, f"{buf}: load of {version} over {b.version}, unread by {sorted(map(str, b.left))}"
        old, b.version = b.version, ("landing", version)

        def land():
            b.version = old
            b.write(version)
            self.bars[bar].arrive()

        self.loads.append(land)

    def issue(self, thread, fn):
        self.mma.setdefault(thread, []).append(fn)
        self.count.setdefault(thread, [0, 0])[0] += 1

    def commit(self, thread, bar):
        self.commits.setdefault(thread, []).append((self.count.get(thread, [0, 0])[0], bar))
        self.settle(thread)

    def settle(self, thread):
        done = self.count.get(thread, [0, 0])[1]
        ready = [b for n, b in self.commits.get(thread, []) if n <= done]
        self.commits[thread] = [(n, b) for n, b in self.commits.get(thread, []) if n > done]
        for b in ready:
            self.bars[b].arrive()

    def execute(self, thread):
        self.mma[thread].pop(0)()
        self.count[thread][1] += 1
        self.settle(thread)

    def wait(self, bar, parity):
        b = self.bars[bar]
        return lambda: b.done(parity & 1)

    def read(self, buf, version, who):
        self.bufs[buf].read(version, who)

    def run(self, max_steps=400_000):
        agents = self.agents()
        waits, done = [None] * len(agents), [False] * len(agents)
        slow = {}   # in each run some agents and units are far slower than the others
        speed = lambda c: slow.setdefault(c if c[0] != "load" else c[0], self.rng.choice((1.0, 1.0, 0.3, 0.02)))  # noqa: E731
        for _ in range(max_steps):
            choices = [("agent", i) for i in range(len(agents)) if not done[i] and (waits[i] is None or waits[i]())]
            choices += [("mma", t) for t, q in self.mma.items() if q]
            choices += [("load", i) for i in range(len(self.loads))]
            if not choices:
                assert all(done), "deadlock"
                assert not any(self.commits.values())
                return
            what, i = self.rng.choices(choices, [speed(c) for c in choices])[0]
            if what == "agent":
                try:
                    waits[i] = next(agents[i])
                except StopIteration:
                    done[i] = True
            elif what == "mma":
                self.execute(i)
            else:
                self.loads.pop(i)()
        raise AssertionError("step limit")

    def ring_loader(self, name, stages, full, empty):
        for seq in range(len(self.blocks)):
            st = seq % stages
            yield self.wait(f"{empty}{st}", (seq // stages & 1) ^ 1)
            self.load(f"{name}{st}", seq, f"{full}{st}")


STEP = lambda: True  # noqa: E731 - a place where an agent can be interrupted


# ------------------------------------------------------------------ forward

class Forward(Model):
    """one_buffer: the maps take one score buffer in turn (d = 128), else one each (d = 64)."""

    def __init__(self, items, seed, mutation=None, one_buffer=True):
        super().__init__(items, seed, mutation)
        self.one, self.ks = one_buffer, 2
        for name, count, n in (("QFull", 1, 2), ("QEmpty", 1, 2), ("SFull", 1, 2), ("SFree", 4, 2), ("PFull", 4, 2),
                               ("PvDone", 1, 2), ("KFull", 1, 2), ("KEmpty", 1, 2), ("VFull", 1, 2), ("VEmpty", 1, 2),
                               ("LxBar", 2, 4), ("OFull", 1, None), ("OFree", 8, None)):
            self.bar(name, count, n)
        for i in range(2):
            self.buf(f"Q{i}", lambda k: {("S", m, self.first[k] + j) for m in (0, 1) for j in range(items[k])})
            self.buf(f"K{i}", lambda s: {("S", m, s) for m in (0, 1)})
            self.buf(f"V{i}", lambda s: {("PV", m, s) for m in (0, 1)})
            self.buf(f"P{i}", lambda v, i=i: {("PV", i, v)}, 4)
            self.buf(f"S{i}", lambda v: {4 * v[1] + q for q in range(4)})
            # O_m of a block: the next block's product goes on from it, an item's last is read by all
            self.buf(f"O{i}", lambda s: set(WARPS) if self.last(s) else set())
            for q in range(4):
                for m in (0, 1):   # the row sums of map m, read by the other map's warp
                    self.buf(f"L{i}{m}{q}", lambda k, m=m, q=q: {4 * (1 - m) + q})

    def last(self, seq):
        k, j = self.blocks[seq]
        return j + 1 == self.items[k]

    def agents(self):
        return [self.q_and_k(), self.ring_loader("V", 2, "VFull", "VEmpty"), self.s_issuer(), self.pv_issuer()] + \
               [self.softmax(w) for w in WARPS]

    def q_and_k(self):
        seq = 0
        for k, n in enumerate(self.items):
            qb = k & 1
            yield self.wait(f"QEmpty{qb}", (k >> 1 & 1) ^ 1)
            self.load(f"Q{qb}", k, f"QFull{qb}")
            for _ in range(n):
                st = seq % 2
                yield self.wait(f"KEmpty{st}", (seq // 2 & 1) ^ 1)
                self.load(f"K{st}", seq, f"KFull{st}")
                seq += 1

    def s_issuer(self):
        seq = 0
        for k, n in enumerate(self.items):
            qb = k & 1
            yield self.wait(f"QFull{qb}", k >> 1)
            for j in range(n):
                st = seq % 2
                yield self.wait(f"KFull{st}", seq // 2)
                for m in (0, 1):
                    of = 1 - m if self.one else m
                    ph = seq if self.one and m == 1 else seq - 1
                    if ph >= 0 and self.mutation != "no_sfree":
                        yield self.wait(f"SFree{of}", ph)

                    def s(m=m, seq=seq, k=k, st=st, qb=qb):
                        self.read(f"Q{qb}", k, ("S", m, seq))
                        self.read(f"K{st}", seq, ("S", m, seq))
                        self.bufs["S0" if self.one else f"S{m}"].write((seq, m))

                    self.issue("s", s)
                    if m == (0 if self.mutation == "early_kempty" else 1):
                        self.commit("s", f"KEmpty{st}")
                    if m == 1 and j + 1 == n:
                        self.commit("s", f"QEmpty{qb}")
                    self.commit("s", f"SFull{m}")
                seq += 1

    def pv_issuer(self):
        seq = 0
        for k, n in enumerate(self.items):
            if k > 0 and self.mutation != "no_ofree":
                yield self.wait("OFree", k - 1)
            for j in range(n):
                st = seq % 2
                yield self.wait(f"VFull{st}", seq // 2)
                for m in (0, 1):
                    yield self.wait(f"PFull{m}", seq)

                    def pv(m=m, seq=seq, st=st):
                        self.read(f"V{st}", seq, ("PV", m, seq))
                        self.read(f"P{m}", seq, ("PV", m, seq))
                        self.bufs[f"O{m}"].write(seq)

                    self.issue("pv", pv)
                    self.commit("pv", f"PvDone{m}")
                self.commit("pv", f"VEmpty{st}")
                if j + 1 == n:
                    self.commit("pv", "OFull")
                seq += 1

    def softmax(self, w):
        m, quad, seq = w >> 2, w & 3, 0
        for k, n in enumerate(self.items):
            for j in range(n):
                yield self.wait(f"SFull{m}", seq)
                self.read("S0" if self.one else f"S{m}", (seq, m), w)
                yield STEP
                self.bars[f"SFree{m}"].arrive()
                if seq > 0 and self.mutation != "no_pvdone":
                    yield self.wait(f"PvDone{m}", seq - 1)
                else:
                    yield STEP
                if j > 0 and self.rng.random() < 0.5:   # a raised maximum: O is read and written
                    self.read(f"O{m}", seq - 1, w)
                    yield STEP
                    self.read(f"O{m}", seq - 1, w)
                self.bufs[f"P{m}"].write(seq)
                yield STEP
                self.bars[f"PFull{m}"].arrive()
                seq += 1
                yield STEP
            x = k & 1
            self.bufs[f"L{x}{m}{quad}"].write(k)
            yield STEP
            self.bars[f"LxBar{quad}"].arrive()
            if self.mutation != "no_lx":
                yield self.wait(f"LxBar{quad}", k)
            yield self.wait("OFull", k)
            self.read(f"L{x}{1 - m}{quad}", k, w)
            for mm in (0, 1):
                self.read(f"O{mm}", seq - 1, w)
                yield STEP
            self.bars["OFree"].arrive()


# ------------------------------------------------------------------ dQ

class Dq(Model):
    """stages: of K and of V, 2 at d = 128 and 4 at d = 64."""

    def __init__(self, items, seed, mutation=None, stages=2):
        super().__init__(items, seed, mutation)
        self.ks = stages
        for name, count, n in (("FixFull", 1, None), ("FixEmpty", 1, None), ("KFull", 1, stages), ("KEmpty", 1, stages),
                               ("VFull", 1, stages), ("VEmpty", 1, stages), ("SFull", 1, 2), ("SFree", 4, 2),
                               ("DsFull", 4, 2), ("DsDone", 1, 2), ("PFull", 1, None), ("PFree", 8, None), ("OFull", 1, None)):
            self.bar(name, count, n)
        self.buf("Fix", lambda k: {(op, self.first[k] + j) for op in ("S0", "S1", "dP") for j in range(items[k])})
        for i in range(stages):
            self.buf(f"K{i}", lambda s: {(op, s) for op in ("S0", "S1", "dQ0", "dQ1")})
            self.buf(f"V{i}", lambda s: {("dP", s)})
        self.buf("S", lambda v: {4 * v[1] + q for q in range(4)})
        self.buf("dP", lambda s: set(WARPS))
        for m in (0, 1):
            self.buf(f"dS{m}", lambda s, m=m: {(f"dQ{m}", s)}, 4)
            self.buf(f"dQ{m}", lambda s, m=m: {4 * m + q for q in range(4)} if self.last(s) else set())

    last = Forward.last

    def agents(self):
        return [self.fix_and_k(), self.ring_loader("V", self.ks, "VFull", "VEmpty"), self.s_issuer(), self.dq_issuer()] + \
               [self.elementwise(w) for w in WARPS]

    def fix_and_k(self):
        seq = 0
        for k, n in enumerate(self.items):
            yield self.wait("FixEmpty", (k & 1) ^ 1)
            self.load("Fix", k, "FixFull")
            for _ in range(n):
                st = seq % self.ks
                yield self.wait(f"KEmpty{st}", (seq // self.ks & 1) ^ 1)
                self.load(f"K{st}", seq, f"KFull{st}")
                seq += 1

    def s_issuer(self):
        seq = 0
        for k, n in enumerate(self.items):
            yield self.wait("FixFull", k)
            for j in range(n):
                st, ph = seq % self.ks, seq // self.ks
                yield self.wait(f"KFull{st}", ph)
                for m in (0, 1):
                    if (m == 1 or seq > 0) and self.mutation != "no_sfree":
                        yield self.wait(f"SFree{1 - m}", seq if m == 1 else seq - 1)

                    def s(m=m, seq=seq, k=k, st=st):
                        self.read("Fix", k, (f"S{m}", seq))
                        self.read(f"K{st}", seq, (f"S{m}", seq))
                        self.bufs["S"].write((seq, m))

                    self.issue("s", s)
                    self.commit("s", f"SFull{m}")
                yield self.wait(f"VFull{st}", ph)
                if seq > 0 and self.mutation != "no_pfree":
                    yield self.wait("PFree", seq - 1)
                if self.mutation == "early_fix_empty" and j + 1 == n:
                    self.commit("s", "FixEmpty")

                def dp(seq=seq, k=k, st=st):
                    self.read("Fix", k, ("dP", seq))
                    self.read(f"V{st}", seq, ("dP", seq))
                    self.bufs["dP"].write(seq)

                self.issue("s", dp)
                self.commit("s", f"VEmpty{st}")
                if j + 1 == n and self.mutation != "early_fix_empty":
                    self.commit("s", "FixEmpty")
                self.commit("s", "PFull")
                seq += 1

    def dq_issuer(self):
        seq = 0
        for n in self.items:
            for j in range(n):
                st = seq % self.ks
                for m in (0, 1):
                    yield self.wait(f"DsFull{m}", seq)

                    def dq(m=m, seq=seq, st=st):
                        self.read(f"K{st}", seq, (f"dQ{m}", seq))
                        self.read(f"dS{m}", seq, (f"dQ{m}", seq))
                        self.bufs[f"dQ{m}"].write(seq)

                    self.issue("q", dq)
                    self.commit("q", f"DsDone{m}")
                self.commit("q", f"KEmpty{st}")
                if j + 1 == n:
                    self.commit("q", "OFull")
                seq += 1

    def elementwise(self, w):
        m, seq = w >> 2, 0
        for k, n in enumerate(self.items):
            for _ in range(n):
                yield self.wait(f"SFull{m}", seq)
                self.read("S", (seq, m), w)
                yield STEP
                self.bars[f"SFree{m}"].arrive()
                yield self.wait("PFull", seq)
                if seq > 0 and self.mutation != "no_dsdone":
                    yield self.wait(f"DsDone{m}", seq - 1)
                self.read("dP", seq, w)
                yield STEP
                self.bars["PFree"].arrive()
                self.bufs[f"dS{m}"].write(seq)
                yield STEP
                self.bars[f"DsFull{m}"].arrive()
                seq += 1
            yield self.wait("OFull", k)
            self.read(f"dQ{m}", seq - 1, w)


# ------------------------------------------------------------------ dK, dV

class Dkv(Model):
    """qs, os: stages of Q and of dO, 3 and 1 at d = 128, 4 and 4 at d = 64."""

    def __init__(self, items, seed, mutation=None, qs=3, os=1):
        super().__init__(items, seed, mutation)
        self.qs, self.os = qs, os
        for name, count, n in (("FixFull", 1, None), ("FixEmpty", 1, None), ("QFull", 1, qs), ("QEmpty", 1, qs),
                               ("DoFull", 1, os), ("DoEmpty", 1, os), ("LFull", 1, None), ("LEmpty", 8, None),
                               ("DFull", 1, None), ("DEmpty", 8, None), ("SFull", 1, 2), ("SFree", 8, 2), ("PFull", 1, None),
                               ("DsFull", 8, None), ("DsDone", 1, None), ("OFull", 1, None)):
            self.bar(name, count, n)
        self.buf("Fix", lambda k: {(op, self.first[k] + j) for op in ("S0", "S1", "dP") for j in range(items[k])})
        for i in range(qs):
            self.buf(f"Q{i}", lambda s: {(op, s) for op in ("S0", "S1", "dK1", "dK2")})
        for i in range(os):
            self.buf(f"Do{i}", lambda s: {(op, s) for op in ("dP", "dV")})
        self.buf("Lse", lambda s: set(WARPS))
        self.buf("D", lambda s: set(WARPS))
        self.buf("S", lambda v: set(WARPS))
        # dP^T's columns: read by the warps, each of which then stores its parts of P^T and dS_1^T over
        # what it has read; the next dP may come when dV and dK_1 have read those
        self.buf("dP", lambda s: set(WARPS) | {("dV", s), ("dK1", s)})
        self.buf("PT", lambda s: {("dV", s)}, 8)
        self.buf("dS1", lambda s: {("dK1", s)}, 8)
        self.buf("dS2", lambda s: {("dK2", s)}, 8)
        for acc in ("dV", "dK1", "dK2"):
            self.buf(acc, lambda s: set(WARPS) if self.last(s) else set())

    last = Forward.last

    def agents(self):
        return [self.fix_and_q(), self.ring_loader("Do", self.os, "DoFull", "DoEmpty"), self.vectors(), self.issuer()] + \
               [self.elementwise(w) for w in WARPS]

    def fix_and_q(self):
        seq = 0
        for k, n in enumerate(self.items):
            yield self.wait("FixEmpty", (k & 1) ^ 1)
            self.load("Fix", k, "FixFull")
            for _ in range(n):
                st = seq % self.qs
                yield self.wait(f"QEmpty{st}", (seq // self.qs & 1) ^ 1)
                self.load(f"Q{st}", seq, f"QFull{st}")
                seq += 1

    def vectors(self):
        for seq in range(len(self.blocks)):
            yield self.wait("LEmpty", (seq & 1) ^ 1)
            self.load("Lse", seq, "LFull")
            yield self.wait("DEmpty", (seq & 1) ^ 1)
            self.load("D", seq, "DFull")

    def issuer(self):
        mut = self.mutation
        issue = lambda fn: self.issue("m", fn)  # noqa: E731
        commit = lambda bar: self.commit("m", bar)  # noqa: E731
        q_full = lambda i: self.wait(f"QFull{i % self.qs}", i // self.qs)  # noqa: E731
        do_full = lambda i: self.wait(f"DoFull{i % self.os}", i // self.os)  # noqa: E731

        def s(i, m):
            def fn():
                self.read("Fix", self.blocks[i][0], (f"S{m}", i))
                self.read(f"Q{i % self.qs}", i, (f"S{m}", i))
                self.bufs["S"].write((i, m))
            issue(fn)
            commit(f"SFull{m}")

        def dp(i):
            def fn():
                self.read("Fix", self.blocks[i][0], ("dP", i))
                self.read(f"Do{i % self.os}", i, ("dP", i))
                self.bufs["dP"].write(i)
            issue(fn)
            commit("PFull")

        def product(acc, a, b, i):
            def fn():
                self.read(b, i, (acc, i))
                self.read(a, i, (acc, i))
                if acc != "dK2":   # the operand lies in dP's columns
                    self.read("dP", i, (acc, i))
                self.bufs[acc].write(i)
            issue(fn)

        i = 0
        for k, n in enumerate(self.items):
            yield self.wait("FixFull", k)
            yield q_full(i)
            yield do_full(i)
            if i > 0:
                yield self.wait("SFree1", i - 1)
            s(i, 0)
            dp(i)
            yield self.wait("SFree0", i)
            s(i, 1)
            if n == 1:
                commit("FixEmpty")
            for j in range(n):
                more = j + 1 < n
                if more:
                    yield q_full(i + 1)
                    if mut != "no_sfree":
                        yield self.wait("SFree1", i)
                    s(i + 1, 0)
                yield self.wait("DsFull", i)
                if mut == "dp_before_dv" and more:
                    yield do_full(i + 1) if self.os > 1 else STEP
                    dp(i + 1)
                product("dV", "PT", f"Do{i % self.os}", i)
                commit(f"DoEmpty{i % self.os}")
                if more:
                    yield self.wait("SFree0", i + 1)
                    s(i + 1, 1)
                if mut == "early_fix_empty" and more and j + 2 == n:
                    commit("FixEmpty")
                product("dK1", "dS1", f"Q{i % self.qs}", i)
                if more and mut != "dp_before_dv":
                    yield do_full(i + 1)
                    dp(i + 1)
                if more and j + 2 == n and mut != "early_fix_empty":
                    commit("FixEmpty")
                product("dK2", "dS2", f"Q{i % self.qs}", i)
                commit("DsDone")
                commit(f"QEmpty{i % self.qs}")
                if not more:
                    commit("OFull")
                i += 1

    def elementwise(self, w):
        mut, seq = self.mutation, 0
        for k, n in enumerate(self.items):
            for _ in range(n):
                for m in (0, 1):
                    yield self.wait(f"SFull{m}", seq)
                    if m == 0:
                        yield self.wait("LFull", seq)
                    self.read("S", (seq, m), w)
                    yield STEP
                    self.bars[f"SFree{m}"].arrive()
                    if mut == "early_lempty" and m == 0:
                        self.read("Lse", seq, w)
                        self.bars["LEmpty"].arrive()
                        yield STEP
                self.read("Lse", seq, w)
                yield STEP
                if mut != "early_lempty":
                    self.bars["LEmpty"].arrive()
                yield self.wait("PFull", seq)
                yield self.wait("DFull", seq)
                self.read("dP", seq, w)
                self.read("D", seq, w)
                yield STEP
                self.bufs["PT"].write(seq)
                self.bufs["dS1"].write(seq)
                if seq > 0 and mut != "no_dsdone":
                    yield self.wait("DsDone", seq - 1)
                else:
                    yield STEP
                self.bufs["dS2"].write(seq)
                yield STEP
                self.bars["DEmpty"].arrive()
                self.bars["DsFull"].arrive()
                seq += 1
            yield self.wait("OFull", k)
            for acc in ("dK1", "dK2", "dV"):
                self.read(acc, seq - 1, w)
                yield STEP


KERNELS = {
    "forward_d128": (Forward, dict(one_buffer=True)), "forward_d64": (Forward, dict(one_buffer=False)),
    "dq_d128": (Dq, dict(stages=2)), "dq_d64": (Dq, dict(stages=4)),
    "dkv_d128": (Dkv, dict(qs=3, os=1)), "dkv_d64": (Dkv, dict(qs=4, os=4)),
}


def cases(n, seed):
    rng = random.Random(seed)
    for trial in range(n):
        yield [rng.randint(1, 5) for _ in range(rng.randint(1, 5))], trial


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_no_deadlock_and_no_stale_data(kernel):
    model, kw = KERNELS[kernel]
    for items, trial in cases(300, 1):
        model(items, trial, **kw).run()


PLANTED = [
    ("forward_d128", "no_sfree"), ("forward_d64", "no_sfree"), ("forward_d128", "no_ofree"), ("forward_d128", "no_pvdone"),
    ("forward_d64", "early_kempty"), ("forward_d128", "no_lx"),
    ("dq_d128", "no_sfree"), ("dq_d128", "no_pfree"), ("dq_d64", "no_dsdone"), ("dq_d128", "early_fix_empty"),
    ("dkv_d128", "no_sfree"), ("dkv_d64", "dp_before_dv"), ("dkv_d128", "no_dsdone"), ("dkv_d128", "early_fix_empty"),
    ("dkv_d64", "early_lempty"),
]


@pytest.mark.parametrize("kernel,mutation", PLANTED)
def test_planted_mistakes_are_caught(kernel, mutation):
    model, kw = KERNELS[kernel]
    caught = 0
    for items, trial in cases(100, 2):
        try:
            model(items, trial, mutation, **kw).run()
        except AssertionError:
            caught += 1
    assert caught >= 10, f"{mutation}: caught in only {caught} of 100"
