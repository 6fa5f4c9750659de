"""The barriers of the tensor-core key-weights kernel, as a model on the CPU.

The kernel's roles (keys, queries, two MMA warps, two softmax groups per key
tile) meet at mbarriers, whose waits know a phase by its parity alone: a wait for
a phase passes as well while the phase two before it is the last one complete.
So every wait has to be for a phase whose predecessor the waiting role knows to be
complete, and nothing may be written while something still reads it. The model
walks the roles and the asynchronous work (loads land in any order, an MMA
warp's commits in its own) in random orders, with roles held back for long, and
checks the phase behind every wait that passes and what every slot holds when it
is read.

Four rules of the kernel keep it sound. Without them the model has to fail, so that
it is known to see the mistake (what the commit of a query slot guards, the
drain guards too, so the first is left out together with the second):
  keys     both MMA warps see and free every tile of the key ring
  queries  query slots are freed by a commit, also where a block has no second
           key tile
  scores   a score buffer belongs to one key tile and one of its groups
  drain    an MMA warp without keys in a block first waits for its groups
"""
import random

import pytest

RULES = ("keys", "queries", "scores", "drain")
SCORE_BUFS, RING, RECORDS, JOINS = 4, 16, 4, 2


class Broken(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.done = 0  # phases complete

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.done += 1
            self.left = self.count


class Cta:
    """One CTA's walk over `items`: (query tiles, [key tiles of each block])."""

    def __init__(self, items, qslots, kslots, rules):
        self.items, self.qs, self.ks, self.rules = items + [(None, [])], qslots, kslots, rules
        bars = lambda n, count: [Bar(count) for _ in range(n)]  # noqa: E731
        self.kfull, self.kfree = bars(kslots, 1), bars(kslots, 2 if "keys" in rules else 1)
        self.qfull, self.qfree = bars(qslots, 1), bars(qslots, 2)
        self.sfull, self.sfree = bars(SCORE_BUFS, 2), bars(SCORE_BUFS, 1)
        self.ifull, self.ifree = bars(RECORDS, 1), bars(RECORDS, 1 + 2 + 4)
        self.jfull, self.jfree = bars(2 * JOINS, 1), bars(2 * JOINS, 1)
        self.K, self.Q = [None] * kslots, [None] * qslots
        self.S, self.stats = [None] * SCORE_BUFS, [None] * RING
        self.products = []   # operands of products in flight: (kind, slot, value)
        self.entries = []    # entries of the statistics' ring in use
        self.pending = {"k": [], "q": [], "0": [], "1": []}

    # -- what the roles share
    def wait(self, bar, phase, what):
        while (bar.done - 1) & 1 != phase & 1:
            yield
        if bar.done - 1 != phase:
            raise Broken(f"{what}: waited for phase {phase}, passed at {bar.done - 1}")

    def holds(self, what, at, want):
        if at != want:
            raise Broken(f"{what} holds {at}, not {want}")

    def land(self, kind, slots, slot, value, bar):
        if any(p[:2] == (kind, slot) for p in self.products):
            raise Broken(f"{kind}[{slot}] is overwritten while products read it")
        slots[slot] = value
        bar.arrive()

    # -- the roles
    def keys(self):
        kn = 0
        for it, (count, blocks) in enumerate(self.items):
            rec = it % RECORDS
            if it >= RECORDS:
                yield from self.wait(self.ifree[rec], it // RECORDS - 1, "item free")
            self.ifull[rec].arrive()
            yield
            if count is None:
                return
            for x, ktiles in enumerate(blocks if count else []):
                for a in range(ktiles):
                    s = kn % self.ks
                    if kn >= self.ks:
                        yield from self.wait(self.kfree[s], kn // self.ks - 1, "key slot free")
                    self.pending["k"].append(
                        lambda s=s, v=(it, x, a): self.land("K", self.K, s, v, self.kfull[s]))
                    kn += 1
                    yield

    def queries(self):
        n = 0
        for it, (count, _) in enumerate(self.items):
            rec = it % RECORDS
            yield from self.wait(self.ifull[rec], it // RECORDS, "item, queries")
            self.ifree[rec].arrive()
            if count is None:
                return
            for _ in range(count):
                s = n % self.qs
                if n >= self.qs:
                    yield from self.wait(self.qfree[s], n // self.qs - 1, "query slot free")
                for e in self.entries:
                    if e % RING == n % RING:
                        raise Broken(f"statistics {e} are overwritten by {n} while in use")
                self.stats[n % RING] = n
                self.pending["q"].append(
                    lambda s=s, v=n: self.land("Q", self.Q, s, v, self.qfull[s]))
                n += 1
                yield

    def mma(self, a):
        r = self.rules
        n = pairs = kn = si = 0
        used = [0] * SCORE_BUFS

        def pass_tile(i):
            yield from self.wait(self.kfull[i % self.ks], i // self.ks, "other keys")
            self.kfree[i % self.ks].arrive()

        for it, (count, blocks) in enumerate(self.items):
            rec = it % RECORDS
            yield from self.wait(self.ifull[rec], it // RECORDS, "item, mma")
            if count is None:
                return
            for x, ktiles in enumerate(blocks if count else []):
                last = x + 1 == len(blocks)
                if "keys" in r and a > 0:
                    yield from pass_tile(kn)
                if "drain" in r and a >= ktiles:
                    for buf in (a, a + 2):
                        if used[buf]:
                            yield from self.wait(self.sfree[buf], used[buf] - 1, "drain")
                for j in range(count):
                    s = (n + j) % self.qs
                    yield from self.wait(self.qfull[s], (n + j) // self.qs, "queries")
                    if a < ktiles:
                        k, sj = (kn + a) % self.ks, si + j * ktiles + a
                        if j == 0:
                            yield from self.wait(self.kfull[k], (kn + a) // self.ks, "keys")
                        buf = a + 2 * ((pairs + j) & 1) if "scores" in r else sj % SCORE_BUFS
                        use = used[buf] if "scores" in r else sj // SCORE_BUFS
                        used[buf] += 1
                        if use:
                            yield from self.wait(self.sfree[buf], use - 1, "scores free")
                        self.sfull[buf].arrive()
                        ops = [("K", k, (it, x, a)), ("Q", s, n + j)]
                        self.products += ops

                        def done(ops=ops, buf=buf, v=(it, x, a, j), k=k, s=s, end=j + 1 == count,
                                 last=last):
                            for kind, slot, want in ops:
                                self.holds(kind, (self.K if kind == "K" else self.Q)[slot], want)
                                self.products.remove((kind, slot, want))
                            self.S[buf] = v
                            self.sfull[buf].arrive()
                            if end:
                                self.kfree[k].arrive()
                            if last:
                                self.qfree[s].arrive()
                        self.pending[str(a)].append(done)
                    elif last and "queries" in r:
                        self.pending[str(a)].append(self.qfree[s].arrive)
                    elif last:
                        self.qfree[s].arrive()
                    yield
                if "keys" in r and a + 1 < ktiles:
                    yield from pass_tile(kn + 1)
                kn += ktiles
                si += count * ktiles
                pairs += count
            n += count
            self.ifree[rec].arrive()
            yield

    def softmax(self, a, group):
        own = "scores" in self.rules
        n = pairs = si = joins = used = 0
        for it, (count, blocks) in enumerate(self.items):
            rec = it % RECORDS
            yield from self.wait(self.ifull[rec], it // RECORDS, "item, softmax")
            if count is None:
                return
            for x, ktiles in enumerate(blocks):
                if a < ktiles:
                    for j in range(((pairs if own else n) ^ group) & 1, count, 2):
                        sj = si + j * ktiles + a
                        buf = a + 2 * group if own else sj % SCORE_BUFS
                        yield from self.wait(self.sfull[buf], used if own else sj // SCORE_BUFS,
                                             "scores")
                        used += 1
                        self.entries.append(n + j)
                        for _ in range(2):
                            yield
                            self.holds("scores", self.S[buf], (it, x, a, j))
                            self.holds("statistics", self.stats[(n + j) % RING], n + j)
                        self.entries.remove(n + j)
                        self.sfree[buf].arrive()
                        yield
                    jb = joins % JOINS * 2 + a
                    if group == 0:
                        if joins >= JOINS:
                            yield from self.wait(self.jfree[jb], joins // JOINS - 1, "join free")
                        self.jfull[jb].arrive()
                    else:
                        yield from self.wait(self.jfull[jb], joins // JOINS, "join")
                        self.jfree[jb].arrive()
                    joins += 1
                    yield
                si += count * ktiles
                pairs += count
            n += count
            self.ifree[rec].arrive()
            yield


def walk(items, qslots, kslots, rules, rng, steps=100000):
    """Runs one random order; raises Broken."""
    c = Cta(items, qslots, kslots, rules)
    roles = {"keys": c.keys(), "queries": c.queries(), "mma0": c.mma(0), "mma1": c.mma(1)}
    roles.update({f"soft{a}{g}": c.softmax(a, g) for a in range(2) for g in range(2)})
    names = list(roles) + list(c.pending)
    weight = {x: 10 ** rng.uniform(-3, 0) for x in names}
    for _ in range(steps):
        if not roles:
            return
        if rng.random() < 0.01:  # another role is held back
            weight[rng.choice(names)] = 10 ** rng.uniform(-3, 0)
        live = [x for x in names if x in roles or c.pending.get(x)]
        x = rng.choices(live, [weight[y] for y in live])[0]
        if x in c.pending:
            work = c.pending[x]
            work.pop(rng.randrange(len(work)) if x in "kq" else 0)()
            continue
        try:
            next(roles[x])
        except StopIteration:
            del roles[x]
    raise Broken("a wait never passes: " + ", ".join(roles))


def shapes(rng):
    """A CTA's items as the host cuts them."""
    kind = rng.randrange(4)
    if kind <= 1:  # runs of key blocks, whose query tiles stay in shared memory
        count = rng.choice([1, 2, 3, 4])
        blocks = [2] * rng.choice([0, 1, 2, 4]) + [rng.choice([1, 2])]
        items = [(count, blocks)] * rng.randrange(2, 7)
        if rng.random() < 0.3:  # (a run that nobody sees)
            items.insert(rng.randrange(len(items)), (0, blocks))
        return items, *((2, 4) if count <= 2 else (4, 2))
    if kind == 2:  # one block per item, many tiles; the last block may have one key tile
        return [(rng.randrange(24), [rng.choice([1, 2])]) for _ in range(rng.randrange(2, 7))], 3, 3
    return [(rng.randrange(3), [rng.choice([1, 2])]) for _ in range(rng.randrange(2, 9))], 2, 4


def test_no_order_of_the_roles_breaks_it():
    rng = random.Random(1)
    for _ in range(300):
        walk(*shapes(rng), RULES, rng)


@pytest.mark.parametrize("without,made", [
    (("keys",), None), (("scores",), None),
    (("drain",), ([(20, [2]), (24, [1])] * 2, 3, 3)),
    (("queries", "drain"), ([(2, [2, 1])] * 5, 2, 4)),
])
def test_the_rules_are_needed(without, made):
    rng = random.Random(2)
    rules = tuple(r for r in RULES if r not in without)
    with pytest.raises(Broken):
        for _ in range(3000):
            walk(*(made or shapes(rng)), rules, rng)
