"""A model of the barriers of the tile kernel of kvq_chunk_attention_nvfp4
(csrc/chunk_attention.cu): its roles as coroutines that take random times,
its mbarriers with the parity that the hardware tests beside the phase that
each wait means.  A wait that passes before its phase is complete ("early"),
one whose phase has been followed by another before it looked ("missed"), and
shared memory that is written while somebody still reads it are faults.

Fillers, product warps and segments are the kernel's; two warps stand for the
four of each softmax group.  Each product warp's products end in order, at
random times."""
import heapq
import random

WARPS = 2


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.arrived, self.done = name, count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived = 0
            self.done += 1

    def passes(self, phase):
        return (self.done & 1) != (phase & 1)


class Model:
    """segments: (two query tiles?, KV tiles) of one thread block's share;
    empties, announcements: barriers per K or V tile ring, and per ring of
    segments."""

    def __init__(self, segments, seed, empties, announcements, slow=None,
                 tail=30, own_first=True):
        self.rng = random.Random(seed)
        self.segs, self.slow, self.tail = segments, slow or {}, tail
        self.depth, self.ann = empties, announcements
        self.own_first = own_first
        self.now, self.queue, self.pushed, self.faults = 0, [], 0, []
        self.bars = {}
        for name, n, count in (
                ("k_full", 2, 4), ("v_full", 2, 4), ("q_full", 2, WARPS),
                ("s_full", 2, 1), ("p_full0", 2, WARPS),
                ("p_full1", 2, WARPS), ("p_done", 2, 1), ("o_done", 2, 1),
                ("turn", 2, 1), ("k_empty", empties, 2),
                ("v_empty", empties, 2), ("o_free", 1, 2 * WARPS),
                ("segment", announcements, 2)):
            for i in range(n):
                self.bars[name, i] = Bar(f"{name}[{i}]", count)
        self.tiles, self.first = [], []
        for s, (_, n) in enumerate(segments):
            self.first.append(len(self.tiles))
            self.tiles += [(s, i) for i in range(n)]
        self.K, self.V = [{}, {}], [{}, {}]     # quarters: tile held
        self.product_end = [0, 0]
        self.query_used = [0, 0]
        self.valid_read, self.over, self.joining = {}, {}, {}

    # --- time ---------------------------------------------------------------
    def push(self, t, item):
        self.pushed += 1
        heapq.heappush(self.queue, (t, self.pushed, item))

    def takes(self, who, base):
        x = base * self.rng.uniform(.3, 1.5) * self.slow.get(who, 1)
        if self.rng.random() < .04:
            x += self.rng.uniform(0, self.tail)
        return ("time", x)

    def wait(self, name, i, phase):
        return ("wait", self.bars[name, i], phase)

    def arrive(self, name, i, times=1):
        for _ in range(times):
            self.bars[name, i].arrive()

    def issue(self, m, done, base):
        self.product_end[m] = max(self.now, self.product_end[m]) + \
            base * self.rng.uniform(.5, 2)
        self.push(self.product_end[m], ("product", done))

    def run(self):
        for m in range(2):
            for w in range(WARPS):
                self.push(0, (f"softmax {m}.{w}", self.softmax(m, w)))
            self.push(0, (f"product {m}", self.product(m)))
        for f in range(6):
            self.push(0, (f"filler {f}", self.filler(f)))
        parked, pairs = [], {}
        while self.queue or parked or pairs:
            if not self.queue:
                self.faults.append(("stuck", [
                    (who, bar.name, phase, bar.done)
                    for who, _, bar, phase in parked]))
                break
            self.now, _, (who, role) = heapq.heappop(self.queue)
            op = role() if callable(role) else next(role, None)
            if op and op[0] == "time":
                self.push(self.now + op[1], (who, role))
            elif op and op[0] == "wait":
                parked.append((who, role, op[1], op[2]))
            elif op and op[0] == "pair":
                pairs.setdefault(op[1], []).append((who, role))
                if len(pairs[op[1]]) == 2:
                    for x in pairs.pop(op[1]):
                        self.push(self.now + .01, x)
            still = []
            for who, role, bar, phase in parked:
                if bar.passes(phase):
                    if bar.done <= phase:
                        self.faults.append(("early", bar.name, who, phase))
                    self.push(self.now + self.rng.uniform(.02, .3),
                              (who, role))
                else:
                    if bar.done >= phase + 2:
                        self.faults.append(("missed", bar.name, who, phase))
                    still.append((who, role, bar, phase))
            parked = still
            if len(self.faults) > 6:
                break
        return self.faults

    def check(self, ok, *fault):
        if not ok:
            self.faults.append(fault)

    # --- roles --------------------------------------------------------------
    def announced(self, s):
        """The wait for segment s (s > 0)."""
        return self.wait("segment", s % self.ann, (s - 1) // self.ann)

    def softmax(self, m, w):
        who, tiles = f"softmax {m}.{w}", [0, 0]
        for s, (two, n) in enumerate(self.segs):
            if s:
                yield self.announced(s)
            if m == 0 or two:
                self.check(not self.query_used[m], "query written", who, s)
                yield self.takes(who, 1.5)
                self.arrive("q_full", m)
            cnt, first = tiles[m], 0 if two else m
            for kt in range(first, n, 1 if two else 2):
                yield self.wait("s_full", m, cnt)
                for half in range(2):
                    yield self.takes(who, .5)
                    if self.rng.random() < .1 and (kt > first or half):
                        # done over: every product of the slot so far
                        yield (self.wait("p_done", m, cnt) if half else
                               self.wait("o_done", m, cnt - 1))
                        yield self.takes(who, .5)
                    if half:
                        t = self.first[s] + kt
                        self.valid_read[t] = self.valid_read.get(t, 0) + 1
                    self.arrive(f"p_full{half}", m)
                cnt += 1
            tiles[0] += n if two else (n + 1) // 2
            tiles[1] += n if two else n // 2
            if two:
                yield self.wait("o_done", m, cnt - 1)
            else:
                yield from self.join(m, w, n, tiles, s)
            yield self.takes(who, 1.0)
            self.over[s] = self.over.get(s, 0) + 1
            self.arrive("o_free", 0)
        yield self.announced(len(self.segs))

    def join(self, m, w, n, tiles, s):
        who = f"softmax {m}.{w}"
        # its own slot's last product, the joint barrier, the other slot's
        # (or, as the model's alternative, both before it)
        own = 1 if m == 1 and n > 1 else 0
        if not self.own_first:
            own = 0
        yield self.wait("o_done", own, tiles[own] - 1)
        if n > 1 and not self.own_first:
            yield self.wait("o_done", 1, tiles[1] - 1)
        self.check(not self.joining.get((w, 1 - m)), "sums written", who, s)
        yield ("pair", w, 2)
        if n > 1 and self.own_first:
            yield self.wait("o_done", 1 - own, tiles[1 - own] - 1)
        self.joining[w, m] = True
        yield self.takes(who, .3)
        self.joining[w, m] = False

    def product(self, m):
        who, cnt, queries, weights, turns = f"product {m}", 0, 0, 0, 0
        for s, (two, n) in enumerate(self.segs):
            step, first, q = (1, 0, m) if two else (2, m, 0)
            yield self.wait("q_full", 0, s)
            if q == 1:
                yield self.wait("q_full", 1, queries)
            for i in range(first, n + step, step):
                pv, qk = i >= first + step, i < n
                tv, tk = cnt + i - step, cnt + i
                if pv:
                    yield self.wait("v_full", tv & 1, tv >> 1)
                    yield self.wait("p_full0", m, weights)
                    if i == first + step and s:
                        yield self.wait("o_free", 0, s - 1)
                    self.holds(self.V, tv, "V at its product")
                    self.issue(m, lambda: self.arrive("p_done", m), .25)
                if qk:
                    yield self.wait("k_full", tk & 1, tk >> 1)
                if two and pv:
                    if turns + m:
                        yield self.wait("turn", m, turns + m - 1)
                    turns += 1
                if pv:
                    yield self.wait("p_full1", m, weights)
                    weights += 1

                    def v_done(tv=tv, two=two):
                        self.holds(self.V, tv, "V under its product")
                        self.arrive("o_done", m)
                        self.arrive("v_empty", tv % self.depth, 2 - two)
                    self.issue(m, v_done, .25)
                    if two and not qk:
                        self.arrive("turn", 1 - m)
                if qk:
                    self.query_used[q] += 1

                    def k_done(tk=tk, two=two, q=q):
                        self.query_used[q] -= 1
                        self.holds(self.K, tk, "K under its product")
                        self.arrive("s_full", m)
                        self.arrive("k_empty", tk % self.depth, 2 - two)
                    self.issue(m, k_done, .5)
                    if two and pv:
                        self.arrive("turn", 1 - m)
                yield self.takes(who, .1)
                if i == first:
                    yield self.takes(who, .3)
                    self.check(m or s < 3 or
                               self.over.get(s - 3, 0) == 2 * WARPS,
                               "segment ring written", who, s)
                    self.arrive("segment", (s + 1) % self.ann)
            queries += two
            cnt += n

    def holds(self, stages, tile, what):
        held = stages[tile & 1]
        self.check([held.get(x) for x in range(4)] == [tile] * 4, what, tile,
                   dict(held))

    def filler(self, f):
        who = f"filler {f}"
        for j in range(f, 8 * len(self.tiles), 6):
            t, job = divmod(j, 8)
            v = job >= 4
            if t >= 2:  # the tile before in this stage has been multiplied
                yield self.wait("v_empty" if v else "k_empty",
                                (t - 2) % self.depth, (t - 2) // self.depth)
            yield self.takes(who, .4)
            (self.V if v else self.K)[t & 1][job & 3] = t
            s, i = self.tiles[t]
            if not v and t >= 8:
                need = WARPS * (2 if self.segs[self.tiles[t - 8][0]][0] else 1)
                self.check(self.valid_read.get(t - 8, 0) >= need,
                           "valid ring written", who, t)
            if v and i == 0 and s >= 4:
                self.check(self.over.get(s - 4, 0) == 2 * WARPS,
                           "NaN ring written", who, s)
            self.arrive("v_full" if v else "k_full", t & 1)


def random_run(seed, empties, announcements, own_first=True):
    """A random share under random delays, some roles much slower."""
    rng = random.Random(seed)
    if rng.random() < .3:
        segs = [(False, 1)] * rng.randint(1, 14)
    else:
        segs = [(rng.random() < .5, rng.choice([1, 1, 2, 3, 4, 5, 9, 12]))
                for _ in range(rng.randint(1, 14))]
    names = [f"softmax {m}.{w}" for m in range(2) for w in range(WARPS)]
    names += ["product 0", "product 1"] + [f"filler {f}" for f in range(6)]
    slow = {x: rng.choice([3, 10, 30]) for x in names if rng.random() < .15}
    return Model(segs, seed, empties, announcements, slow,
                 rng.choice([0, 5, 30, 100]), own_first).run()
