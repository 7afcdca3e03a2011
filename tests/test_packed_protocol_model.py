"""A discrete-event model of the barrier protocols of csrc/packed_attn.cu and
csrc/packed_bwd.cu (CPU only), in the style of the other kernels' models, with
one difference: a wait polls.  A role may be held up for long at any point, also
between a barrier's completion and its own look at it, and then looks again; so
a wait that can be overtaken by a second phase ends in a deadlock here.

Hazard checks: no slot is reloaded before its readers have finished, no product
reads a slot that does not hold its own tiles, no column of tensor memory is
overwritten before it was read, every product reads what its own step wrote,
outputs are read after the last product, and every role finishes.  Planted
mistakes (a wait left out, one barrier for two regions, a signal behind the commit
that it must precede) are caught.
"""
import heapq
import itertools
import random

import pytest

from test_ring_protocol_model import Hazard


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.tx, self.phase = name, count, count, 0, 0

    def passed(self, parity):
        return (self.phase & 1) != parity

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        if self.pending < 0:
            raise Hazard("more arrivals than the count on " + self.name)
        self.settle()

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count


class Sim:
    """Roles are generators of actions:
        ("delay", cycles)          ("wait", barrier, parity)   ("arrive", barrier)
        ("copy", barrier, landed)  bytes that land later, `landed` called then
        ("mma", cycles, finished)  on the in-order pipe, `finished` called at its end
        ("commit", barrier)        arrives once the pipe has got there"""

    def __init__(self, seed, sluggish):
        self.rng, self.now, self.queue, self.n = random.Random(seed), 0, [], itertools.count()
        self.sluggish, self.pipe_free, self.roles, self.done = sluggish, 0, {}, set()
        self.asleep = []  # (role, barrier, parity) that polled in vain

    def at(self, delay, fn):
        heapq.heappush(self.queue, (self.now + delay, next(self.n), fn))

    def pause(self):
        if self.rng.random() < self.sluggish:
            return self.rng.randint(500, 20000)
        return self.rng.randint(5, 150)

    def step(self, role):
        try:
            act = next(self.roles[role])
        except StopIteration:
            self.done.add(role)
            return
        kind = act[0]
        if kind == "wait":
            self.poll(role, act[1], act[2])
            return
        if kind == "arrive":
            act[1].arrive()
            self.wake()
        elif kind == "copy":
            bar, landed = act[1], act[2]
            bar.arrive(tx=1)

            def land(bar=bar, landed=landed):
                landed()
                bar.tx -= 1
                bar.settle()
                self.wake()
            self.at(self.rng.randint(6000, 30000) if self.rng.random() < 0.1 else self.rng.randint(300, 3000), land)
        elif kind == "mma":
            self.pipe_free = max(self.now, self.pipe_free) + act[1]
            self.at(self.pipe_free - self.now, act[2])
        elif kind == "commit":
            def arrive(bar=act[1]):
                bar.arrive()
                self.wake()
            self.at(max(0, self.pipe_free - self.now) + self.rng.randint(1, 50), arrive)
        delay = act[1] if kind == "delay" else 0
        self.at(delay + self.pause(), lambda: self.step(role))

    def poll(self, role, bar, parity):
        if bar.passed(parity):
            self.at(self.pause(), lambda: self.step(role))
        else:
            self.asleep.append((role, bar, parity))

    def wake(self):  # every wait looks again, each at its own time
        again, self.asleep = self.asleep, []
        for role, bar, parity in again:
            if bar.passed(parity):
                self.at(self.pause(), lambda r=role, b=bar, p=parity: self.poll(r, b, p))
            else:
                self.asleep.append((role, bar, parity))

    def run(self):
        for role in self.roles:
            self.at(self.pause(), lambda role=role: self.step(role))
        while self.queue:
            self.now, _, fn = heapq.heappop(self.queue)
            fn()
        if len(self.done) != len(self.roles):
            raise Hazard("deadlock: " + ", ".join("%s at %s" % (r, b.name) for r, b, _ in self.asleep))


def nothing():
    pass


class Slots:
    """Ring slots: what each holds, whether it has landed, readers to come."""

    def __init__(self, name, count):
        self.name, self.count, self.held = name, count, [None] * count

    def load(self, x, what, readers):
        h = self.held[x % self.count]
        if h and h["readers"]:
            raise Hazard("%s slot of %s reloaded with %s, %s still reads it" % (self.name, h["what"], what, h["readers"]))
        self.held[x % self.count] = dict(what=what, landed=False, readers=set(readers))

    def land(self, x):
        self.held[x % self.count]["landed"] = True

    def use(self, x, what):
        h = self.held[x % self.count]
        if not h or h["what"] != what or not h["landed"]:
            raise Hazard("%s read where the %s slot holds %s" % (what, self.name, h))

    def free(self, x, what, reader):
        h = self.held[x % self.count]
        if h["what"] == what:
            h["readers"].discard(reader)


class Columns:
    """Columns of tensor memory, per group of warps and warp: what they hold
    and whether it has been taken."""

    def __init__(self, name, warps):
        self.name, self.warps = name, [dict(what=None, taken=True) for _ in range(warps)]

    def put(self, what, w=None):
        for c in self.warps if w is None else [self.warps[w]]:
            if not c["taken"]:
                raise Hazard("%s written over %s of %s" % (what, c["what"], self.name))
            c.update(what=what, taken=False)

    def see(self, what, w=None):
        for c in self.warps if w is None else [self.warps[w]]:
            if c["what"] != what:
                raise Hazard("%s read from %s, which holds %s" % (what, self.name, c["what"]))

    def take(self, what, w=None):
        self.see(what, w)
        for c in self.warps if w is None else [self.warps[w]]:
            c["taken"] = True


# ---- dK, dV: CTA = 128 keys --------------------------------------------------------
def dkdv(sim, n, tails, wrong=None):
    """n steps; `tails`: the steps whose query tile is partial."""
    NR = 2
    full = [Barrier("full%d" % s, 1) for s in range(NR)]
    x_free, s_ready, dp_ready, st_issued, own, fix_go, fixed = (
        Barrier(x, 1) for x in ("x_free", "s_ready", "dp_ready", "st_issued", "own", "fix_go", "fixed"))
    dp_read, ds_ready = (Barrier(x, 8) for x in ("dp_read", "ds_ready"))
    p_ready = [Barrier("p_ready%d" % r, 8) for r in range(1 if wrong == "one p_ready" else 2)]
    done = Barrier("done", 2)
    ring = Slots("Q/dO", NR)
    region = [Columns("region %d" % r, 8) for r in range(2)]   # S^T, then P^T; or dP^T
    region_ds = [Columns("dS^T of region %d" % r, 8) for r in range(2)]
    log = dict(dv=0, dk=0, s=-1)

    def p_of(p):  # the barrier of step p's P^T and its parity
        return (p_ready[0], p & 1) if wrong == "one p_ready" else (p_ready[p & 1], (p >> 1) & 1)

    def copies():
        yield ("copy", own, nothing)
        for p in range(n):
            if p >= NR and wrong != "no wait of the copies":
                yield ("wait", x_free, (p - NR) & 1)
            ring.load(p, p, ["S", "dP", "dV", "dK"] + list(range(8)))
            yield ("copy", full[p % NR], lambda p=p: ring.land(p))

    def tail():
        for i, _ in enumerate(tails):
            yield ("wait", fix_go, i & 1)
            yield ("delay", 300)
            yield ("arrive", fixed)

    def issuer():
        seen = 0
        yield ("wait", own, 0)
        for p in range(n):
            yield ("wait", full[p % NR], (p // NR) & 1)
            if p in tails:
                yield ("arrive", fix_go)
                yield ("wait", fixed, seen & 1)
                seen += 1
            if p > 0 and wrong != "dp_read":
                yield ("wait", dp_read, (p - 1) & 1)
            ring.use(p, p)
            region[p & 1].put(("S", p))
            log["s"] = p
            yield ("mma", 512, lambda p=p: ring.free(p, p, "S"))
            if wrong == "late st_issued":
                yield ("commit", s_ready)
                yield ("arrive", st_issued)
            else:
                yield ("arrive", st_issued)
                yield ("commit", s_ready)
            if p > 0 and wrong != "x_free of dP":
                yield ("wait", x_free, (p - 1) & 1)
            ring.use(p, p)
            region[1 - (p & 1)].put(("dP", p))
            yield ("mma", 512, lambda p=p: ring.free(p, p, "dP"))
            yield ("commit", dp_ready)
        yield ("commit", done)

    def accumulations():
        for p in range(n):
            yield ("wait", *p_of(p))
            region[p & 1].see(("P", p))
            ring.use(p, p)
            yield ("mma", 512, lambda p=p: (region[p & 1].take(("P", p)), ring.free(p, p, "dV"), log.update(dv=p + 1)))
            if p + 1 < n and wrong != "no st_issued":
                yield ("wait", st_issued, (p + 1) & 1)
                if log["s"] < p + 1:
                    raise Hazard("dK of step %d queued in front of the next S^T" % p)
            if wrong != "ds_ready":
                yield ("wait", ds_ready, p & 1)
            region_ds[p & 1].see(("dS", p))
            ring.use(p, p)
            yield ("mma", 512, lambda p=p: (region_ds[p & 1].take(("dS", p)), ring.free(p, p, "dK"), log.update(dk=p + 1)))
            yield ("commit", x_free)
        yield ("commit", done)

    def warp(w):
        for p in range(n):
            yield ("wait", s_ready, p & 1)
            region[p & 1].take(("S", p), w)
            ring.use(p, p)  # the rows' lse
            yield ("delay", sim.rng.randint(200, 1500))
            region[p & 1].put(("P", p), w)
            yield ("arrive", p_of(p)[0])
            yield ("wait", dp_ready, p & 1)
            region[1 - (p & 1)].take(("dP", p), w)
            yield ("arrive", dp_read)
            ring.use(p, p)  # and D
            yield ("delay", sim.rng.randint(100, 800))
            ring.free(p, p, w)
            region_ds[p & 1].put(("dS", p), w)
            yield ("arrive", ds_ready)
        yield ("wait", done, 0)
        if log["dv"] != n or log["dk"] != n:
            raise Hazard("written after %s of %d steps" % (log, n))

    sim.roles = dict(copies=copies(), tail=tail(), issuer=issuer(), accumulations=accumulations(),
                     **{"warp%d" % w: warp(w) for w in range(8)})


# ---- dQ: CTA = 128 query rows --------------------------------------------------------
def dq(sim, n, tail, exact, wrong=None):
    """n key steps; `exact`: a first sweep sums D; `tail`: the last tile is partial."""
    NK, NV = 3, 2
    lead = n if exact and n > 1 else 0
    nt = lead + n
    kfull, kempty = ([Barrier("%s%d" % (x, s), 1) for s in range(NK)] for x in ("kfull", "kempty"))
    vfull, vempty = ([Barrier("%s%d" % (x, s), 1) for s in range(NV)] for x in ("vfull", "vempty"))
    sd_ready, x_free, bar_q, bar_do, fix_go, fixed = (
        Barrier(x, 1) for x in ("sd_ready", "x_free", "q", "do", "fix_go", "fixed"))
    read, x_ready, sums = (Barrier(x, 8) for x in ("read", "x_ready", "sums"))
    own, done = Barrier("own", 4), Barrier("done", 2)
    s_ready = [Barrier("s_ready%d" % b, 1) for b in range(2)]
    s_read = [Barrier("s_read%d" % b, 8) for b in range(2)]
    kring, vring = Slots("K", NK), Slots("V", NV)
    S, ACC, DP, DS = (Columns(x, 8) for x in ("S", "the sum", "dP", "dS"))
    log = dict(acc=0, dsum=0)

    def copies():
        kring.load(2, "dO", range(4, 8))
        yield ("copy", bar_do, lambda: kring.land(2))
        yield ("copy", bar_q, nothing)
        for p in range(nt):
            if p >= NK and wrong != "kempty":
                yield ("wait", kempty[p % NK], ((p - NK) // NK) & 1)
            if p == 2 and wrong != "own":
                yield ("wait", own, 0)
            kring.load(p, p, ["S"] if p < lead else ["S", "dQ"])
            yield ("copy", kfull[p % NK], lambda p=p: kring.land(p))
            if p >= NV:
                yield ("wait", vempty[p % NV], ((p - NV) // NV) & 1)
            vring.load(p, p, ["dP"])
            yield ("copy", vfull[p % NV], lambda p=p: vring.land(p))

    def tail_warp():
        if tail:
            yield ("wait", fix_go, 0)
            yield ("delay", 300)
            kring.use(nt - 1, nt - 1)
            yield ("arrive", fixed)

    def issuer():
        yield ("wait", own, 0)
        yield ("wait", bar_q, 0)
        for p in range(lead):
            yield ("wait", kfull[p % NK], (p // NK) & 1)
            if p >= 2:
                yield ("wait", s_read[p & 1], ((p >> 1) - 1) & 1)
            kring.use(p, p)
            (ACC if p & 1 else S).put(("S", p))
            yield ("mma", 512, lambda p=p: kring.free(p, p, "S"))
            yield ("commit", s_ready[p & 1])
            yield ("commit", kempty[p % NK])
            yield ("wait", vfull[p % NV], (p // NV) & 1)
            if p > 0:
                yield ("wait", read, (p - 1) & 1)
            vring.use(p, p)
            DP.put(("dP", p))
            yield ("mma", 512, lambda p=p: vring.free(p, p, "dP"))
            yield ("commit", sd_ready)
            yield ("commit", vempty[p % NV])
        for p in range(lead, nt):
            yield ("wait", kfull[p % NK], (p // NK) & 1)
            yield ("wait", vfull[p % NV], (p // NV) & 1)
            if p > 0 and wrong != "read":
                yield ("wait", read, (p - 1) & 1)
            if tail and p == nt - 1:
                yield ("arrive", fix_go)
                yield ("wait", fixed, 0)
            kring.use(p, p)
            vring.use(p, p)
            S.put(("S", p))
            DP.put(("dP", p))
            yield ("mma", 1024, lambda p=p: (kring.free(p, p, "S"), vring.free(p, p, "dP")))
            yield ("commit", sd_ready)
            yield ("commit", vempty[p % NV])
        yield ("commit", done)

    def accumulations():
        for p in range(lead, nt):
            yield ("wait", x_ready, (p - lead) & 1)
            DS.see(("dS", p))
            kring.use(p, p)
            if p == lead:
                ACC.put("dQ")  # its columns held the first sweep's odd scores
            yield ("mma", 512, lambda p=p: (DS.take(("dS", p)), kring.free(p, p, "dQ"), log.update(acc=log["acc"] + 1)))
            yield ("commit", x_free)
            yield ("commit", kempty[p % NK])
        yield ("commit", done)

    def warp(w):
        if w >= 4:  # group 1 takes dO to tensor memory
            yield ("wait", bar_do, 0)
            kring.use(2, "dO")
            yield ("delay", 200)
            kring.free(2, "dO", w)
            yield ("arrive", own)
        if exact and n:
            for p in range(n):
                if lead:
                    yield ("wait", s_ready[p & 1], (p >> 1) & 1)
                    (ACC if p & 1 else S).take(("S", p), w)
                    yield ("arrive", s_read[p & 1])
                    yield ("delay", sim.rng.randint(100, 900))
                yield ("wait", sd_ready, p & 1 if lead else 0)
                if lead:
                    DP.take(("dP", p), w)
                    yield ("arrive", read)
                else:
                    S.see(("S", p), w)
                    DP.see(("dP", p), w)
                yield ("delay", sim.rng.randint(50, 300))
            log["dsum"] += 1
            yield ("arrive", sums)
            yield ("wait", sums, 0)
            if log["dsum"] != 8:
                raise Hazard("D read before both halves were in")
        for p in range(n):
            yield ("wait", sd_ready, (lead + p) & 1)
            S.take(("S", lead + p), w)
            DP.take(("dP", lead + p), w)
            yield ("arrive", read)
            yield ("delay", sim.rng.randint(200, 1500))
            if p > 0 and wrong != "x_free":
                yield ("wait", x_free, (p - 1) & 1)
            DS.put(("dS", lead + p), w)
            yield ("arrive", x_ready)
        yield ("wait", done, 0)
        if log["acc"] != n:
            raise Hazard("written after %d of %d steps" % (log["acc"], n))

    if n:
        sim.roles = dict(copies=copies(), tail=tail_warp(), issuer=issuer(), accumulations=accumulations(),
                         **{"warp%d" % w: warp(w) for w in range(8)})


# ---- forward: two query tiles that walk the same keys, entry after entry ------------
def forward(sim, entries, ring_slots, split, wrong=None):
    """entries: (steps of tile 0, of tile 1, the walk ends in a partial key tile);
    split: one entry only."""
    R, INFO = ring_slots, 4
    full, empty = ([Barrier("%s%d" % (x, s), 1) for s in range(R)] for x in ("full", "empty"))
    q, q_free, s_bar, o_bar = ([Barrier("%s%d" % (x, t), 1) for t in range(2)] for x in ("q", "q_free", "s", "o"))
    p_bar = [Barrier("p%d" % t, 4) for t in range(2)]
    info = [Barrier("info%d" % b, 1) for b in range(INFO)]
    info_free = [Barrier("info_free%d" % b, 11) for b in range(INFO)]
    fix_go, fixed = Barrier("fix_go", 1), Barrier("fixed", 1)
    ring, Q = Slots("stage", R), [Slots("Q%d" % t, 1) for t in range(2)]
    S, O = ([Columns("%s%d" % (x, t), 4) for t in range(2)] for x in "SO")
    board = [None] * INFO
    last_entry = len(entries)  # its place says that the list has ended

    def take(it):  # as published; every warp but the finder's arrives
        yield ("wait", info[it % INFO], (it // INFO) & 1)
        if board[it % INFO] != it:
            raise Hazard("entry %d read where %s stands" % (it, board[it % INFO]))
        yield ("arrive", info_free[it % INFO])
        return entries[it] if it < last_entry else None

    def finder():
        for it in itertools.count():
            if it >= INFO and wrong != "info_free":
                yield ("wait", info_free[it % INFO], (it // INFO - 1) & 1)
            board[it % INFO] = it
            yield ("arrive", info[it % INFO])
            if split or it == last_entry:
                return

    def steps(e):
        return max(e[0], e[1]) if e else 0

    def copies():
        x, nq, joined = 0, [0, 0], False

        def stage(v, k):
            nonlocal x
            if x >= R and wrong != "empty":
                yield ("wait", empty[x % R], (x // R - 1) & 1)
            ring.load(x, (v, k), (["v"] if v else []) + (["k"] if k else []))
            yield ("copy", full[x % R], lambda x=x: ring.land(x))
            x += 1

        e = yield from take(0)
        it = 0
        while e is not None:
            n = steps(e)
            if n:
                if not joined:
                    yield from stage(None, (it, 0))
                for t in range(2):
                    if e[t]:
                        if nq[t] > 0 and wrong != "q_free":
                            yield ("wait", q_free[t], (nq[t] - 1) & 1)
                        nq[t] += 1
                        Q[t].load(0, it, range(e[t]))
                        yield ("copy", q[t], lambda t=t: Q[t].land(0))
                for j in range(1, n):
                    yield from stage((it, j - 1), (it, j))
            nxt = None
            if not split:
                nxt = yield from take(it + 1)
            joined = n > 0 and steps(nxt) > 0
            if n:
                yield from stage((it, n - 1), (it + 1, 0) if joined else None)
            e, it = nxt, it + 1

    def products():
        c, nq, tails, did, joined = 0, [0, 0], 0, [0, 0], False
        holds = {}  # what the copies put into each stage, for the checks alone

        def scores(t, x, it, j):
            Q[t].use(0, it)
            ring.use(x, holds[x])
            assert holds[x][1] == (it, j)
            S[t].put(("S", it, j))
            yield ("mma", 512, lambda t=t, it=it, j=j: Q[t].free(0, it, j))
            yield ("commit", s_bar[t])

        def first(t, e, it, x):
            if e[t]:
                yield ("wait", q[t], nq[t] & 1)
                nq[t] += 1
                yield from scores(t, x, it, 0)
                if e[t] == 1:
                    yield ("commit", q_free[t])

        e = yield from take(0)
        it = 0
        while e is not None:
            n = steps(e)
            if not n:
                if split:
                    return
                it += 1
                e = yield from take(it)
                continue
            if not joined:
                holds[c] = (None, (it, 0))
                yield ("wait", full[c % R], (c // R) & 1)
                for t in range(2):
                    yield from first(t, e, it, c)
                yield ("mma", 0, lambda c=c: ring.free(c, holds[c], "k"))
                yield ("commit", empty[c % R])
            nxt = None
            for i in range(n):
                last = i == n - 1
                if last and not split:
                    nxt = yield from take(it + 1)
                joined = last and steps(nxt) > 0
                x = c + i + 1
                holds[x] = ((it, i), (it, i + 1) if not last else (it + 1, 0) if joined else None)
                yield ("wait", full[x % R], (x // R) & 1)
                if e[2] and last:
                    yield ("arrive", fix_go)
                    if wrong != "fixed":
                        yield ("wait", fixed, tails & 1)
                    tails += 1
                for t in range(2):
                    if i < e[t]:
                        yield ("wait", p_bar[t], did[t] & 1)
                        did[t] += 1
                        ring.use(x, holds[x])
                        S[t].see(("P", it, i))
                        if e[2] and last and tails_done[0] != tails:
                            raise Hazard("V read before its tail was zeroed")
                        if i == 0:
                            O[t].put(it)
                        yield ("mma", 512, lambda t=t, it=it, i=i: nothing())
                        S[t].take(("P", it, i))  # what follows on the pipe comes behind it
                        if i + 1 < e[t]:
                            yield from scores(t, x, it, i + 1)
                            if i + 2 == e[t]:
                                yield ("commit", q_free[t])
                        else:
                            yield ("commit", o_bar[t])
                    if joined:
                        yield from first(t, nxt, it + 1, x)
                yield ("mma", 0, lambda x=x: (ring.free(x, holds[x], "k"), ring.free(x, holds[x], "v")))
                yield ("commit", empty[x % R])
            c += n if joined else n + 1
            e, it = nxt, it + 1

    tails_done = [0]

    def tail_warp():
        tails = 0
        e = yield from take(0)
        it = 0
        while e is not None:
            nxt = None
            if not split:
                nxt = yield from take(it + 1)
            if steps(e) and e[2]:
                yield ("wait", fix_go, tails & 1)
                tails += 1
                yield ("delay", 300)
                tails_done[0] = tails
                yield ("arrive", fixed)
            e, it = nxt, it + 1

    def softmax(t, w):
        done = tiles = 0
        for it in itertools.count():
            e = yield from take(it)
            if e is None:
                return
            for i in range(e[t]):
                yield ("wait", s_bar[t], (done + i) & 1)
                S[t].take(("S", it, i), w)
                yield ("delay", sim.rng.randint(300, 2500))
                S[t].put(("P", it, i), w)
                yield ("arrive", p_bar[t])
            done += e[t]
            if e[t]:
                if wrong != "o":
                    yield ("wait", o_bar[t], tiles & 1)
                tiles += 1
                O[t].take(it, w)
            yield ("delay", sim.rng.randint(200, 1500))
            if split:
                return

    sim.roles = dict(copies=copies(), products=products(), tail=tail_warp(), finder=finder(),
                     **{"softmax%d.%d" % (t, w): softmax(t, w) for t in range(2) for w in range(4)})


def simulate(kernel, trial, wrong=None):
    rng = random.Random("%s %d" % (kernel, trial))
    sim = Sim(trial, rng.choice([0.0, 0.02, 0.2]))
    if kernel == "dkdv":
        n = rng.choice([0, 1, 2, 3, 5, 8, 24])
        per = rng.randint(1, max(1, n))
        tails = [p for p in range(n) if p % per == per - 1] if rng.random() < 0.5 else []
        dkdv(sim, n, tails, wrong)
    elif kernel == "dq":
        dq(sim, rng.choice([0, 1, 2, 3, 4, 5, 8, 20]), rng.random() < 0.5, rng.random() < 0.5, wrong)
    else:
        kinds = rng.choice([[0, 1], [1], [1, 2, 3], [0, 1, 2, 6], [4, 9]])
        entries = []
        for _ in range(rng.choice([1, 2, 5, 12])):
            a = rng.choice(kinds)
            b = a if rng.random() < 0.5 else rng.choice(kinds)
            entries.append((a, b, rng.random() < 0.4))
        split = rng.random() < 0.2
        forward(sim, entries[:1] if split else entries, rng.choice([2, 4]), split, wrong)
    sim.run()


@pytest.mark.parametrize("kernel", ["forward", "dq", "dkdv"])
def test_no_hazard(kernel):
    for trial in range(250):
        try:
            simulate(kernel, trial)
        except Hazard as e:
            pytest.fail("%s, trial %d: %s" % (kernel, trial, e))


@pytest.mark.parametrize("kernel,wrong", [
    ("dkdv", "one p_ready"),            # the accumulations may look two phases late
    ("dkdv", "no st_issued"),           # and then so may the copies at x_free
    ("dkdv", "late st_issued"),         # dK in front of the S^T that the groups wait for
    ("dkdv", "no wait of the copies"), ("dkdv", "dp_read"), ("dkdv", "x_free of dP"), ("dkdv", "ds_ready"),
    ("dq", "kempty"), ("dq", "own"), ("dq", "read"), ("dq", "x_free"),
    ("forward", "empty"), ("forward", "q_free"), ("forward", "info_free"), ("forward", "fixed"), ("forward", "o"),
])
def test_planted_mistake_is_caught(kernel, wrong):
    for trial in range(250):
        try:
            simulate(kernel, trial, wrong)
        except Hazard:
            return
    pytest.fail("the model no longer sees it")
