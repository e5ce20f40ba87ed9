"""The protocol of the prefixes' tensor-core kernel (csrc/serving/prefix_tc.cu) as a model on the CPU: one producer, two
issuers of products, two softmax streams, mbarriers that are waited for by the parity of their phase, loads that land in any
order, and a scheduler that lets any of them lag.  Checked at every step: products read the fill they mean, which has landed
and stays until they are done; no barrier gets more arrivals than its phase has room for (a warp's come together); nobody
waits for ever.  The same where a stream's wait gives up and the others see that.

`sent`, `seen`: the two conditions under which a parity tells a phase from the one before last -- a fill is waited for only
once it is known to have been sent; a segment's Q rows follow once both issuers have seen the last segment's.  Without the
first the model fails, as the kernel did: with 5 or 6 slots a slot goes from one stream's fill to the other's."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Wrong(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, n=1, tx=0):
        self.tx += tx
        if n > self.pending:
            raise Wrong("more arrivals than the phase has room for")
        self.pending -= n
        self._turn()

    def land(self):
        self.tx -= 1
        self._turn()

    def done(self, parity):  # the phase of this parity is complete, as far as a parity can say
        return (self.phase & 1) != parity


class Model:
    def __init__(self, slots, segments, rng, sent=True, seen=True, stall=None):
        self.n, self.segs, self.rng, self.use_sent, self.use_seen, self.stall = slots, segments, rng, sent, seen, stall
        self.count = sum(n for n, _ in segments)
        self.full, self.empty = [Bar(1) for _ in range(slots)], [Bar(1) for _ in range(slots)]
        self.S, self.O = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
        self.P, self.Q, self.seen = [Bar(129), Bar(128)], Bar(256), Bar(2)
        self.slot = [None] * slots  # (fill, landed)
        self.sent, self.loads, self.pipe, self.readers = 0, [], [[], []], [0] * slots
        self.named, self.named_turn = 0, 0
        self.abort = False

    # ---- what the products do
    def read(self, fill):
        if self.slot[fill % self.n] != (fill, True):
            raise Wrong(f"a product reads fill {fill} where {self.slot[fill % self.n]} is")

    def issue(self, m, op, fill):
        self.read(fill)
        self.readers[fill % self.n] += 1
        self.pipe[m].append((op, fill))

    def commit(self, m, bar):
        self.pipe[m].append(("commit", bar))

    def complete(self, m):
        op, x = self.pipe[m].pop(0)
        if op == "commit":
            x.arrive()
        else:
            self.read(x)
            self.readers[x % self.n] -= 1

    def land(self):
        f = self.loads.pop(self.rng.randrange(len(self.loads)))
        self.slot[f % self.n] = (f, True)
        self.full[f % self.n].land()

    # ---- the roles; each yields the condition that it waits for
    def wait(self, cond):
        yield lambda: cond() or self.abort
        return cond()

    def wait_full(self, fill):
        if self.use_sent and not (yield from self.wait(lambda: self.sent > fill)):
            return False
        return (yield from self.wait(lambda: self.full[fill % self.n].done((fill // self.n) & 1)))

    def producer(self):
        for f in range(2 * self.count):
            slot, use = f % self.n, f // self.n
            if use > 0 and not (yield from self.wait(lambda: self.empty[slot].done((use - 1) & 1))):
                return
            if self.readers[slot]:
                raise Wrong("a fill is sent where a product reads")
            self.slot[slot] = (f, False)
            self.full[slot].arrive(tx=1)
            self.sent = f + 1
            self.loads.append(f)
            yield lambda: True

    def issuer(self, me):
        j, n_p = 0, [0, 0]
        for seg, (n, by_tile) in enumerate(self.segs):
            ok = yield from self.wait(lambda: self.Q.done(seg & 1))
            if self.use_seen:
                self.seen.arrive()
            if not ok:
                return
            if not by_tile and me == 1:
                for i in range(n):
                    if not (yield from self.wait_full(2 * (j + i) + 1)):
                        return
                    if i + 1 < n and not (yield from self.wait_full(2 * (j + i) + 2)):
                        return
                    self.P[0].arrive()
                    if i + 1 < n and not (yield from self.wait(lambda: self.P[0].done((n_p[0] + i) & 1))):
                        return
            elif not by_tile:
                if not (yield from self.wait_full(2 * j)):
                    return
                for m in range(2):
                    self.issue(0, "S", 2 * j)
                    self.commit(0, self.S[m])
                self.commit(0, self.empty[2 * j % self.n])
                for i in range(n):
                    v, k = 2 * (j + i) + 1, 2 * (j + i) + 2
                    for m in range(2):
                        if not (yield from self.wait(lambda: self.P[m].done((n_p[m] + i) & 1))):
                            return
                        self.issue(0, "PV", v)
                        if i + 1 < n:
                            self.issue(0, "S", k)
                        self.commit(0, (self.S if i + 1 < n else self.O)[m])
                    self.commit(0, self.empty[v % self.n])
                    if i + 1 < n:
                        self.commit(0, self.empty[k % self.n])
            elif me < n:
                for q, i in enumerate(range(me, n, 2)):
                    k = 2 * (j + i)
                    if q == 0:
                        if not (yield from self.wait_full(k)):
                            return
                        self.issue(me, "S", k)
                        self.commit(me, self.S[me])
                        self.commit(me, self.empty[k % self.n])
                    if not (yield from self.wait_full(k + 1)):
                        return
                    if not (yield from self.wait(lambda: self.P[me].done((n_p[me] + q) & 1))):
                        return
                    self.issue(me, "PV", k + 1)
                    if i + 2 >= n:
                        self.commit(me, self.O[me])
                    self.commit(me, self.empty[(k + 1) % self.n])
                    if i + 2 < n:
                        if not (yield from self.wait_full(k + 4)):
                            return
                        self.issue(me, "S", k + 4)
                        self.commit(me, self.S[me])
                        self.commit(me, self.empty[(k + 4) % self.n])
            n_p[0] += (n + 1) // 2 if by_tile else n
            n_p[1] += n // 2 if by_tile else n
            j += n
            yield lambda: True

    def softmax(self, me):
        n_s = n_o = j = 0
        ok = True
        for seg, (n, by_tile) in enumerate(self.segs):
            if seg > 0 and self.use_seen:
                ok = ok and (yield from self.wait(lambda: self.seen.done((seg - 1) & 1)))
            self.abort |= not ok
            for _ in range(4):
                self.Q.arrive(32)
            steps = 0
            for i in range(me if by_tile else 0, n, 2 if by_tile else 1):
                if ok and self.stall == (me, n_s):
                    ok = False  # this stream's wait runs out
                ok = ok and (yield from self.wait(lambda: self.S[me].done(n_s & 1)))
                if not ok:
                    self.abort = True
                    break
                n_s, steps = n_s + 1, steps + 1
                if i + 1 == n and (by_tile or me == 0):  # the prefix's end: V rows behind it are zeroed
                    v = 2 * (j + i) + 1
                    ok = yield from self.wait_full(v)
                    if ok:
                        self.read(v)
                for _ in range(4):
                    self.P[me].arrive(32)
                if by_tile and me == 0:
                    self.P[0].arrive()
                self.abort |= not ok
                yield lambda: True
            if ok and steps:
                ok = yield from self.wait(lambda: self.O[me].done(n_o & 1))
                self.abort |= not ok
                n_o += 1
            j += n
            turn = self.named_turn
            self.named += 1
            if self.named == 2:
                self.named, self.named_turn = 0, turn + 1
            yield lambda: self.named_turn > turn

    def run(self):
        roles = [self.producer(), self.issuer(0), self.issuer(1), self.softmax(0), self.softmax(1)]
        waits = [next(r) for r in roles]
        lag, step = {}, 0
        while any(roles) or self.loads or any(self.pipe):
            moves = [("role", i) for i, r in enumerate(roles) if r and waits[i]()]
            moves += [("land", 0)] * bool(self.loads) + [("pipe", m) for m in (0, 1) if self.pipe[m]]
            if not moves:
                raise Wrong("everybody waits")
            free = [x for x in moves if lag.get(x, 0) <= step] or moves
            kind, i = self.rng.choice(free)
            if self.rng.random() < 0.05:  # somebody falls behind for a while
                lag[self.rng.choice(moves)] = step + self.rng.randrange(200)
            step += 1
            if kind == "land":
                self.land()
            elif kind == "pipe":
                self.complete(i)
            else:
                try:
                    waits[i] = next(roles[i])
                except StopIteration:
                    roles[i] = None


def segments(rng):
    return [(rng.randrange(1, rng.choice([2, 4, 12])), rng.random() < 0.7) for _ in range(rng.randrange(1, 8))]


@pytest.mark.parametrize("slots", [5, 6, 12])
def test_the_protocol(slots):
    for seed in range(400):
        rng = random.Random(seed)
        Model(slots, segments(rng), rng).run()


@pytest.mark.parametrize("slots", [5, 12])
def test_a_wait_that_gives_up(slots):
    for seed in range(300):
        rng = random.Random(seed)
        segs = segments(rng) if seed % 2 else [(1, True)] * rng.randrange(1, 15)
        Model(slots, segs, rng, stall=(rng.randrange(2) if seed % 2 else 0, rng.randrange(4))).run()


@pytest.mark.parametrize("slots", [5, 6])
def test_a_parity_alone_does_not_tell_the_fills_of_two_streams_apart(slots):
    seen = set()
    for seed in range(200):
        rng = random.Random(seed)
        try:
            Model(slots, [(12, True)], rng, sent=False).run()
        except Wrong as e:
            seen.add(str(e).split(" ")[0])
    assert seen


def test_an_issuer_without_tiles_may_fall_behind():
    seen = set()
    for seed in range(300):
        rng = random.Random(seed)
        try:
            Model(12, [(1, True)] * 6 + [(3, True), (2, False)], rng, seen=False).run()
        except Wrong as e:
            seen.add(str(e))
    assert seen


def test_the_kernel_has_both_conditions():
    with open(os.path.join(ROOT, "tree_speculative_decoding_03_gb300", "csrc", "serving", "prefix_tc.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "mbar_init(bar(Bars::kQ), 256);" in text and "mbar_init(bar(Bars::kSeen), 2);" in text
    kernel = text[text.index("prefix_tc_kernel(const"):]
    assert kernel.count("mbar_arrive(bar(Bars::kSeen));") == 1 and "mbar_wait(bar(Bars::kSeen), (seg - 1) & 1, s_abort)" in kernel
    # every wait for a fill but the producer's own at its end goes through wait_sent
    assert len(re.findall(r"mbar_wait\(bar\(Bars::kFull", kernel)) == len(re.findall(r"wait_sent\([^;]*mbar_wait\(bar\(Bars::kFull", kernel)) + 1
    assert kernel.index("mbar_expect_tx(bar(Bars::kFull") < kernel.index("store_release_smem(sent_at, f + 1);")
