"""A model of the prompt kernel's barriers under random schedules (CPU).

Each warp role of the kernel is a generator that waits on and arrives at the same
barriers with the same parities, over random lists of items; asynchronous work (TMA
loads in any order, MMAs in issue order) completes at random moments.  Checked: no
barrier gets more arrivals than a phase takes, every stage, score tile and
probability tile holds what its reader wants, nothing is overwritten before it was
read, and no role waits for ever (a parity wait that is a phase behind does)."""
import random

import pytest

STAGES = {128: 5, 64: 8}


class Bar:
    def __init__(self, count, name):
        self.count, self.pending, self.phase, self.name = count, count, 0, name

    def arrive(self, k=1):
        assert self.pending >= k, f"over-arrival on {self.name} in phase {self.phase}"
        self.pending -= k
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):              # what a try_wait with this parity says
        return (self.phase & 1) != parity


class Ring:
    def __init__(self, n):
        self.n, self.st, self.ph = n, 0, 0

    def next(self, k=1):
        for _ in range(k):
            self.st += 1
            if self.st == self.n:
                self.st = 0
                self.ph ^= 1

    def ahead(self, k):
        r = Ring(self.n)
        r.st, r.ph = self.st, self.ph
        r.next(k)
        return r


class Model:
    def __init__(self, seed, stages):
        self.r = r = random.Random(seed)
        self.N = stages
        self.items = []
        for _ in range(r.randint(1, 7)):
            kinds = ["h"] * r.choice([0, 0, 1, 3]) + ["c"] * r.choice([0, 0, 1, 2, 4]) + ["n"] * r.choice([0, 1, 1, 2]) or ["n"]
            n = len(kinds)
            cnt = r.choice([(n, n), (n, 0), (n - 1, n), (0, n), (n, n)])
            scan = [k == "n" or k == "h" and r.random() < 0.3 for k in kinds]
            self.items.append((kinds, n, cnt, scan, r.random() < 0.3))     # the last: a partial state
        self.bars = {}
        for name, count in [*(("%s%d" % (k, i), 1) for i in (0, 1) for k in ("QFULL", "QEMPTY", "S")), *(("P%d" % i, 5) for i in (0, 1)),
                            *(("O%d" % i, 1) for i in (0, 1)),
                            *(("%s%d" % (k, s), c) for s in range(stages) for k, c in (("F", 4), ("E", 8), ("C", 1), ("W", 4)))]:
            self.bars[name] = Bar(count, name)
        self.stage = [None] * stages
        self.score, self.prob, self.pv = [None, None], [None, None], [None, None]
        self.read = [set(), set()]
        self.mma, self.tma = [], []
        self.q = [None, None]

    def arrive(self, name, k=1):
        self.bars[name].arrive(k)

    def wait(self, name, parity):
        while not self.bars[name].done(parity):
            yield name

    def staging(self, cnt):
        return (cnt[0] > 0) + (cnt[1] > 0)

    def producer(self):
        ring, qn = Ring(self.N), [0, 0]
        for n, (kinds, nt, cnt, scan, part) in enumerate(self.items):
            for j in range(2 * nt + self.staging(cnt)):
                if j == 1:
                    for i in (0, 1):
                        if cnt[i] > 0:
                            yield from self.wait("QEMPTY%d" % i, (qn[i] & 1) ^ 1)
                            qn[i] += 1

                            def loaded(i=i, n=n):
                                self.q[i] = n
                                self.arrive("QFULL%d" % i)
                            self.tma.append(loaded)
                st, ph = ring.st, ring.ph
                ring.next()
                yield from self.wait("E%d" % st, ph ^ 1)
                if j >= 2 * nt:
                    self.stage[st] = ("out", n)
                    self.arrive("F%d" % st, 4)
                elif kinds[j // 2] == "c":
                    self.arrive("C%d" % st)
                else:
                    sc = j & 1 and scan[j // 2]

                    def done(st=st, sc=sc, n=n, j=j):
                        self.stage[st] = (n, j)
                        self.arrive(("C%d" if sc else "F%d") % st)
                    if not sc:
                        self.arrive("F%d" % st, 3)
                    self.tma.append(done)
                yield None

    def gather(self):
        ring, ph = Ring(self.N), [0] * self.N
        for n, (kinds, nt, cnt, scan, part) in enumerate(self.items):
            for j in range(2 * nt):
                st = ring.st
                ring.next()
                cold = kinds[j // 2] == "c"
                if not cold and not (j & 1 and scan[j // 2]):
                    continue
                yield from self.wait("C%d" % st, ph[st])
                ph[st] ^= 1
                if cold:

                    def landed(st=st, n=n, j=j):
                        self.stage[st] = (n, j)
                        self.arrive("F%d" % st)
                    self.tma.append(landed)
                else:
                    assert self.stage[st] == (n, j)
                    self.arrive("F%d" % st)
                yield None
            ring.next(self.staging(cnt))

    def issue_s(self, i, st, n, j):
        def run():
            assert self.stage[st] == (n, 2 * j), ("S reads", self.stage[st], (n, 2 * j))
            assert self.q[i] == n, ("S reads the Q tile of", self.q[i], n)
            if self.score[i] is not None:
                assert all((*self.score[i], w) in self.read[i] for w in range(4)), ("S overwritten", self.score[i])
            self.score[i] = (n, j)
        self.mma += [run, lambda: self.arrive("S%d" % i)]

    def issue_pv(self, i, st, n, j):
        def run():
            assert self.stage[st] == (n, 2 * j + 1), ("PV reads", self.stage[st], (n, 2 * j + 1))
            assert self.prob[i] == (n, j), ("PV reads P", self.prob[i], (n, j))
            self.pv[i] = (n, j)
        self.mma.append(run)

    def issuer(self):
        k, qn, pn = Ring(self.N), [0, 0], [0, 0]
        for n, (kinds, nt, cnt, scan, part) in enumerate(self.items):
            yield from self.wait("F%d" % k.st, k.ph)
            for i in (0, 1):
                if cnt[i] > 0:
                    yield from self.wait("QFULL%d" % i, qn[i] & 1)
                    qn[i] += 1
                    self.issue_s(i, k.st, n, 0)
            self.mma.append(lambda st=k.st: self.arrive("E%d" % st))
            for j in range(nt):
                v, k = k.ahead(1), k.ahead(2)
                for i in (0, 1):
                    if j >= cnt[i]:
                        continue
                    yield from self.wait("P%d" % i, pn[i] & 1)
                    pn[i] += 1
                    self.issue_pv(i, v.st, n, j)
                    if j + 1 < cnt[i]:
                        self.issue_s(i, k.st, n, j + 1)
                    else:
                        self.mma.append(lambda i=i: self.arrive("O%d" % i))
                    yield None
                self.mma.append(lambda st=v.st: self.arrive("E%d" % st))
                if j + 1 < nt:
                    self.mma.append(lambda st=k.st: self.arrive("E%d" % st))
            k.next(self.staging(cnt))

    def relay(self):
        ring, pn = Ring(self.N), [0, 0]

        def full(el):
            yield from self.wait("F%d" % ring.st, ring.ph)
            assert self.stage[ring.st] == el
            self.arrive("E%d" % ring.st, 7)
            ring.next()
        for n, (kinds, nt, cnt, scan, part) in enumerate(self.items):
            yield from full((n, 0))
            for j in range(nt):
                yield from full((n, 2 * j + 1))
                if j + 1 < nt:
                    yield from full((n, 2 * j + 2))
                for i in (0, 1):
                    if j < cnt[i]:
                        if pn[i] > 0:
                            yield from self.wait("P%d" % i, (pn[i] - 1) & 1)
                        pn[i] += 1
                        self.arrive("P%d" % i)
            ring.next(self.staging(cnt))

    def softmax(self, i, w):
        ring, sn, on = Ring(self.N), 0, 0
        for n, (kinds, nt, cnt, scan, part) in enumerate(self.items):
            yield None
            mine = int(i == 1 and cnt[0] > 0)
            ring.next(2 * nt + mine)
            for j in range(cnt[i]):
                yield from self.wait("S%d" % i, sn & 1)
                sn += 1
                if j + 1 == cnt[i] and w == 0:
                    self.arrive("QEMPTY%d" % i)
                assert self.score[i] == (n, j), ("softmax reads S", self.score[i], (n, j))
                yield None
                assert self.score[i] == (n, j)
                self.read[i].add((n, j, w))
                if j > 0:
                    assert self.pv[i] == (n, j - 1), "P written early"
                self.prob[i] = (n, j)
                self.arrive("P%d" % i)
            if cnt[i] > 0:
                yield from self.wait("O%d" % i, on & 1)
                on += 1
                assert self.pv[i] == (n, cnt[i] - 1), "O read early"
                yield from self.wait("F%d" % ring.st, ring.ph)
                for _ in range(3):
                    assert self.stage[ring.st] == ("out", n)
                    yield None
                assert self.stage[ring.st] == ("out", n)
                if part:
                    self.arrive("E%d" % ring.st, 2)
                else:
                    self.arrive("W%d" % ring.st)
            ring.next(self.staging(cnt) - mine)
            yield None

    def writer(self):
        ring, ph = Ring(self.N), [0] * self.N
        for n, (kinds, nt, cnt, scan, part) in enumerate(self.items):
            ring.next(2 * nt)
            for i in (0, 1):
                if cnt[i] == 0:
                    continue
                st = ring.st
                ring.next()
                if part:
                    continue
                yield from self.wait("W%d" % st, ph[st])
                ph[st] ^= 1
                for _ in range(3):
                    assert self.stage[st] == ("out", n)
                    yield None
                self.arrive("E%d" % st, 8)

    def run(self):
        r = self.r
        roles = {"producer": self.producer(), "issuer": self.issuer(), "relay": self.relay(), "writer": self.writer()}
        roles.update({"gather%d" % g: self.gather() for g in range(4)})
        roles.update({"softmax%d%d" % (i, w): self.softmax(i, w) for i in (0, 1) for w in range(4)})
        weight = {k: r.choice([1, 1, 3, 10, 0.2]) for k in roles}
        waits, idle = {}, 0
        while roles:
            moved = False
            if self.tma and r.random() < 0.5:
                self.tma.pop(r.randrange(len(self.tma)))()
                moved = True
            if self.mma and r.random() < 0.5:
                self.mma.pop(0)()
                moved = True
            k = r.choices(list(roles), [weight[x] for x in roles])[0]
            try:
                waits[k] = next(roles[k])
                moved |= waits[k] is None
            except StopIteration:
                del roles[k]
                moved = True
            idle = 0 if moved else idle + 1
            assert idle < 20000, f"waiting for ever: { {k: waits[k] for k in roles} } over {self.items}"
        while self.mma:
            self.mma.pop(0)()


@pytest.mark.parametrize("d", [128, 64])
def test_random_schedules(d):
    for seed in range(150):
        try:
            Model(seed, STAGES[d]).run()
        except AssertionError as e:
            raise AssertionError(f"seed {seed}: {e}") from e
