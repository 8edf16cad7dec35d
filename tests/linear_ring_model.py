"""A model of the hand-over protocol of the linear layer's tensor-core kernel
(block_scaled_bit_bq_b200/csrc/linear.cu, k_linear_mma), run in random order on the CPU.

Agents are the kernel's warps; a step of one is what happens between two yields. Copies and
MMAs are asynchronous: they complete later, copies in any order, MMAs in the order of issue.
Waits go by parity, as the hardware's do. What is checked:

  contents    a slot holds the stage that its reader takes it for, from the issue of an MMA (or
              the read of a chunk of codes) until it completes, and no writer comes early;
  order       the thread that issues an MMA has been handed every write that the MMA reads: the
              writes are known to it through arrivals whose scope takes in both sides (the same
              CTA, or cluster scope on both), or through a copy's bytes on the barrier it waits on;
  the end     with copies that never land, or a wait that gives up early, every agent comes to its
              end, the CTAs that gave up are marked, and a CTA leaves nothing in flight: its copies
              have landed or it waits for them, and the MMAs that it issued or holds are done.
"""

import random


class Barrier:
    def __init__(self, cta, count):
        self.cta, self.count = cta, count
        self.pending, self.tx, self.phase = count, 0, 0
        self.now, self.last = [], []            # (cta or None for a copy, cluster scope, events) of a phase

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count
            self.last, self.now = self.now, []

    def arrive(self, cta, cluster, events):
        assert self.pending > 0, "more arrivals than the barrier counts"
        self.pending -= 1
        self.now.append((cta, cluster, frozenset(events)))
        self._check()

    def expect(self, cta, nbytes, events=()):
        self.tx += nbytes
        self.arrive(cta, False, events)

    def complete(self, nbytes, event):
        self.tx -= nbytes
        self.now.append((None, True, frozenset((event,))))
        self._check()

    def passed(self, parity):
        return (self.phase & 1) != parity


class Agent:
    def __init__(self, cta, name, body):
        self.cta, self.name, self.known = cta, name, set()
        self.gen = body(self)
        self.wait = None                        # (barrier, parity, cluster scope)
        self.answer = None                      # of the wait that ended: False where it gave up

    def learn(self, bar, cluster):
        for cta, far, events in bar.last:
            if cta is None or cta == self.cta or (far and cluster):
                self.known |= events


class Kernel:
    """One CTA (pair: two CTAs) over a number of tiles.

    x_first: in a pair both CTAs' copies of X complete on the first one's barrier (else each
    CTA's on its own, and the second one relays them). arrive_far / wait_far: the second CTA's
    arrivals on the first one's barriers release, and the waits there acquire, at cluster scope.
    lost: a copy that never lands, by its event ("x" or "code", CTA, stage or chunk, part)."""

    GROUPS, WARPS, EPI = 4, 4, 2

    def __init__(self, rng, pair, tiles, blocks, nc, subs, stages, chunks, chunk_parts, x_first=True, arrive_far=True,
                 wait_far=True, lost=None):
        self.rng, self.pair, self.tiles = rng, pair, tiles
        self.kts, self.nc, self.subs, self.NS, self.NC, self.CP = 4 * blocks, nc, subs, stages, chunks, chunk_parts
        self.ts, self.tc = self.kts // subs, self.kts // chunk_parts
        self.x_first, self.arrive_far, self.wait_far = x_first and pair, arrive_far, wait_far
        n = 2 if pair else 1
        self.ctas = [self._cta(r) for r in range(n)]
        self.copies, self.mmas = [], []
        self.lost, self.stop = lost, [False] * n
        self.agents = []
        for r in range(n):
            self.agents += [Agent(r, "x", self.x_warp), Agent(r, "codes", self.codes_warp)]
            self.agents += [Agent(r, f"widen{g}", lambda a, g=g: self.widen_warp(a, g))
                            for g in range(self.GROUPS) for _ in range(self.WARPS)]
            self.agents += [Agent(r, "epilogue", self.epilogue_warp) for _ in range(self.EPI)]
            self.agents.append(Agent(r, "mma", self.mma_warp if r == 0 else self.relay_warp))

    def _cta(self, r):
        full = self.subs * self.WARPS + 1 + (1 if self.pair and r == 0 else 0)
        return {"full": [Barrier(r, full) for _ in range(self.NS)], "empty": [Barrier(r, 1) for _ in range(self.NS)],
                "code_full": [Barrier(r, 1) for _ in range(self.NC)],
                "code_empty": [Barrier(r, self.CP * self.WARPS) for _ in range(self.NC)],
                "acc_full": [Barrier(r, 1) for _ in range(2)],
                "done_bar": Barrier(r, 1),
                "acc_empty": [Barrier(r, self.EPI * (2 if self.pair else 1)) for _ in range(2)],
                "x": [None] * self.NS, "a": [[set() for _ in range(self.subs)] for _ in range(self.NS)],
                "code": [None] * self.NC, "acc": [None, None], "done": -1}

    def live(self, part):
        return part * 64 < self.nc

    def issue(self, copy):
        if copy[5] != self.lost:
            self.copies.append(copy)

    def give_up(self, me):
        self.stop[me.cta] = True

    # ---- agents: yield None to let others run, or a wait (False: it gave up) ----

    def x_warp(self, me):
        c = self.ctas[me.cta]
        s = rnd = 0
        for t in range(self.tiles):
            for kk in range(self.ts):
                if rnd > 0 and not (yield c["empty"][s], (rnd - 1) & 1, False) or self.stop[me.cta]:
                    return self.give_up(me)
                f = t * self.ts + kk
                assert c["done"] >= f - self.NS, "X written over a stage in use"
                n = sum(self.live(kk * self.subs + u) for u in range(self.subs))
                bar = self.ctas[0]["full"][s] if self.x_first else c["full"][s]
                if n == 0:
                    c["x"][s] = f
                c["full"][s].expect(me.cta, n * ((2 - 2 * me.cta) if self.x_first else 1))
                yield
                for u in range(n):
                    self.issue((c, "x", s, f, bar, ("x", me.cta, f, u)))
                    yield
                s += 1
                if s == self.NS:
                    s, rnd = 0, rnd + 1

    def codes_warp(self, me):
        c = self.ctas[me.cta]
        s = rnd = 0
        for n in range(self.tiles * self.tc):
            if rnd > 0 and not (yield c["code_empty"][s], (rnd - 1) & 1, False) or self.stop[me.cta]:
                return self.give_up(me)
            c["code"][s] = None
            c["code_full"][s].expect(me.cta, 1)
            self.issue((c, "code", s, n, c["code_full"][s], ("code", me.cta, n, 0)))
            yield
            s += 1
            if s == self.NC:
                s, rnd = 0, rnd + 1

    def widen_warp(self, me, g):
        c = self.ctas[me.cta]
        s, rnd, k, kp = g // self.subs, 0, g // self.CP, 0
        for t in range(self.tiles):
            for pk in range(g, self.kts, self.GROUPS):
                ok = yield c["code_full"][k], kp, False
                assert not ok or c["code"][k] == t * self.tc + pk // self.CP, "codes of another part"
                yield
                assert not ok or c["code"][k] == t * self.tc + pk // self.CP, "codes written over while read"
                c["code_empty"][k].arrive(me.cta, False, ())
                if not ok or rnd > 0 and not (yield c["empty"][s], (rnd - 1) & 1, False) or self.stop[me.cta]:
                    return self.give_up(me)
                f = t * self.ts + pk // self.subs
                assert c["done"] >= f - self.NS, "codes widened over a stage in use"
                if self.live(pk):
                    e = ("a", me.cta, f, pk % self.subs, id(me))
                    c["a"][s][pk % self.subs].add(e)
                    me.known.add(e)
                yield
                c["full"][s].arrive(me.cta, False, me.known)
                me.known.clear()                # what it wrote is handed over
                s += self.GROUPS // self.subs
                while s >= self.NS:
                    s, rnd = s - self.NS, rnd + 1
                k += self.GROUPS // self.CP
                while k >= self.NC:
                    k, kp = k - self.NC, kp ^ 1

    def relay_warp(self, me):
        c = self.ctas[1]
        s = par = 0
        for _ in range(self.tiles * self.ts):
            if not (yield c["full"][s], par, False) or self.stop[1]:
                self.give_up(me)
                break
            yield
            self.ctas[0]["full"][s].arrive(1, self.arrive_far, me.known)
            me.known.clear()
            s += 1
            if s == self.NS:
                s, par = 0, par ^ 1
        if not (yield c["done_bar"], 0, False):
            self.give_up(me)

    def stage_events(self, s, f):
        """What MMAs of stage f read, with a check that it is there."""
        need = set()
        for c in self.ctas:
            r = c["full"][0].cta
            assert c["x"][s] == f, f"X of stage {c['x'][s]}, not {f}"
            kk = f % self.ts
            for u in range(self.subs):
                if self.live(kk * self.subs + u):
                    need.add(("x", r, f, u))
                    have = [e for e in c["a"][s][u] if e[2] == f]
                    assert len(have) == self.WARPS, "codes not widened"
                    need |= set(have)
        return need

    def mma_warp(self, me):
        if not (yield from self.issue_mmas(me)):
            self.give_up(me)
        self.mmas.append(("done", 0, 0))
        if not (yield self.ctas[0]["done_bar"], 0, False):
            self.give_up(me)

    def issue_mmas(self, me):
        c = self.ctas[0]
        s = par = 0
        for t in range(self.tiles):
            b = t & 1
            if self.stop[0]:
                return False
            if t >= 2:
                if not (yield c["acc_empty"][b], (t // 2 - 1) & 1, self.pair and self.wait_far):
                    return False
                for q in self.ctas:
                    assert ("acc", q["full"][0].cta, t - 2) in me.known, "accumulator reused before its reads are handed over"
            for kk in range(self.ts):
                if not (yield c["full"][s], par, self.pair and self.wait_far):
                    return False
                f = t * self.ts + kk
                need = self.stage_events(s, f)
                missing = need - me.known
                assert not missing, f"not ordered before the MMAs of stage {f}: {sorted(e[:3] for e in missing)[:2]}"
                me.known -= need
                self.mmas.append(("stage", s, f))
                yield
                s += 1
                if s == self.NS:
                    s, par = 0, par ^ 1
            self.mmas.append(("tile", b, t))
            yield
        return True

    def epilogue_warp(self, me):
        c = self.ctas[me.cta]
        for t in range(self.tiles):
            b = t & 1
            if not (yield c["acc_full"][b], (t // 2) & 1, self.pair and self.wait_far) or self.stop[me.cta]:
                return self.give_up(me)
            assert c["acc"][b] == t
            yield
            assert c["acc"][b] == t, "accumulator written over while read"
            far = me.cta != 0
            self.ctas[0]["acc_empty"][b].arrive(me.cta, far and self.arrive_far, {("acc", me.cta, t)})

    # ---- the scheduler ----

    def finish_copy(self):
        c, what, s, f, bar, event = self.copies.pop(self.rng.randrange(len(self.copies)))
        if what == "x":
            c["x"][s] = f
        else:
            c["code"][s] = f
        bar.complete(1, event)

    def finish_mma(self):
        kind, s, f = self.mmas.pop(0)
        if kind == "stage":
            self.stage_events(s, f)             # still there when the MMA has read it
        for c in self.ctas:
            r = c["full"][0].cta
            if kind == "stage":
                c["done"] = f
                for u in range(self.subs):
                    c["a"][s][u] = {e for e in c["a"][s][u] if e[2] != f}
                c["empty"][s].arrive(r, True, ())
            elif kind == "done":
                c["done_bar"].arrive(r, True, ())
            else:
                c["acc"][s] = f
                c["acc_full"][s].arrive(r, True, ())

    def step(self, a):
        """One step of an agent; False where its wait is not over, None where it has ended."""
        if a.wait is not None:
            bar, parity, cluster = a.wait
            if not bar.passed(parity):
                return False
            a.learn(bar, cluster)
            a.wait, a.answer = None, True
        return self.resume(a)

    def resume(self, a):
        try:
            answer, a.answer = a.answer, None
            a.wait = a.gen.send(answer)
        except StopIteration:
            return None
        return True

    def time_out(self, a):
        a.wait, a.answer = None, False
        return self.resume(a)

    def run(self, early=0.0):
        """To the end; early: how likely a step is to end some wait that is not over (a device that
        held the agent up). Returns which CTAs gave up."""
        left = list(self.agents)
        pace = {id(a): self.rng.random() ** 3 + 0.01 for a in left}      # some agents are slow
        idle = 0
        while left:
            x = self.rng.random()
            if x < 0.15 and self.copies:
                self.finish_copy()
            elif x < 0.3 and self.mmas:
                self.finish_mma()
            else:
                a = self.rng.choices(left, [pace[id(a)] for a in left])[0]
                r = self.step(a)
                if r is False and early and self.rng.random() < early:
                    r, early = self.time_out(a), 0.0
                if r is None:
                    left.remove(a)
                idle = 0 if r is not False else idle + 1
                if idle > 200 and not self.copies and not self.mmas and not any(
                        a.wait is None or a.wait[0].passed(a.wait[1]) for a in left):
                    # nothing moves any more: some wait's time is over first
                    assert self.lost or any(self.stop), "no agent gets on: " + ", ".join(a.name for a in left)
                    a = self.rng.choice(left)
                    if self.time_out(a) is None:
                        left.remove(a)
                    idle = 0
        # the CTAs' ends: without a pair each for itself, a pair's after both have come here
        assert not self.mmas, "MMAs in flight as tensor memory is freed"
        for copy in self.copies:
            r = copy[0]["full"][0].cta
            assert self.stop[r], "a CTA that did not give up leaves copies in flight"
        if not any(self.stop):
            assert all(c["done"] == self.tiles * self.ts - 1 for c in self.ctas)
        return self.stop


def random_case(rng, pair):
    """A plan as make_mma_plan makes them: ring sizes, parts to a stage and to a chunk of codes."""
    subs = 2 if pair else rng.choice([1, 2])
    stages = 3 if pair else (4 if subs == 1 else rng.choice([3, 4]))
    blocks = rng.randint(1, 3)
    return dict(pair=pair, tiles=rng.randint(1, 4), blocks=blocks, nc=rng.randint((blocks - 1) * 256 + 1, blocks * 256),
                subs=subs, stages=stages, chunks=rng.choice([2, 4, 6, 8]), chunk_parts=rng.choice([2, 4]))
