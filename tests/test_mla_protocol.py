"""CPU models of the mbarrier protocols of the latent attention's tensor-core kernels: mla_decode_kernel (ql_mla_decode.cu),
mla_expand_kernel and mla_chunk_kernel (ql_mla_chunk.cu), the last two in pairs of CTAs.

Each role of a kernel is a generator that waits, arms, copies, multiplies and arrives as the kernel does; a warp that only arrives beside
others of its kind stands for all of them. Copies land at random later times in any order; products end in the order issued, and a
commit's arrivals come behind them. In a whole run every wait passes in its time. In a broken one a wait runs out while what it waits
for is still on its way: the role records an error, raises its CTA's flag (in a pair the other's, too) and ends, the others see the
flag at some later time. In both the model fails where
* a barrier is armed whose phase is not the copy's own or has an arrival already;
* a barrier gets more arrivals than its count;
* before a wait has run out, a copy goes to a stage that a product still reads, or a product reads a stage that has not landed (later the
  numbers are of no use);
* a CTA ends while a copy into it is in flight;
* no role can move.
"""
import random

import pytest


class Bar:
    """An mbarrier: a phase completes when its arrivals and its expected bytes are all in."""

    def __init__(self, count, name):
        self.count, self.pending, self.tx, self.phase, self.name = count, count, 0, 0, name

    def _complete(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, f"{self.name}: more arrivals than its count"
        self._complete()

    def arm(self, k, nbytes):
        """The expecting arrival of a copy's phase k."""
        assert self.phase == k and self.pending == self.count, f"{self.name}: armed for phase {k} in phase {self.phase}"
        self.tx += nbytes
        self.arrive()

    def bytes(self, n):
        self.tx -= n
        self._complete()


class Stage:
    def __init__(self):
        self.readers, self.parts, self.load = 0, 0, None


class Sim:
    def __init__(self, seed, broken, ctas=1):
        self.rnd = random.Random(seed)
        self.broken, self.flags = broken, [False] * ctas
        self.p_copy, self.p_mma = self.rnd.choice([0.5, 0.1, 0.01]), self.rnd.choice([0.5, 0.1, 0.01])
        self.p_out = self.rnd.choice([0.02, 0.002]) if broken else 0
        self.copies, self.products, self.expired = [], [], 0

    # -- waits
    def wait(self, bar, k, cta):
        while (bar.phase & 1) == (k & 1):
            if self.flags[cta] and self.rnd.random() < 0.3:
                return False
            if self.rnd.random() < self.p_out:
                self.expired += 1
                self.flags[:] = [True] * len(self.flags)
                return False
            yield False
        if not self.broken:
            assert bar.phase == k + 1, f"{bar.name}: phase {k} waited, {bar.phase} completed"
        yield True
        return True

    def alone(self, bar, k):
        while (bar.phase & 1) == (k & 1):
            yield False

    # -- copies and products
    def copy(self, stage, load, parts, land):
        """One of `parts` copies of load `load` into a stage."""
        assert stage.readers == 0 or any(self.flags), f"load {load} over a stage that a product reads"
        if stage.load != load:
            stage.load, stage.parts = load, 0

        def arrived():
            stage.parts += 1
            land()
        self.copies.append(arrived)

    def product(self, stages, after=()):
        """Reads [(stage, load, parts)]; `after` are the commits' arrivals behind it and what was issued before it."""
        for st, load, parts in stages:
            assert (st.load == load and st.parts == parts) or any(self.flags), f"product reads load {load} before it landed"
            st.readers += 1

        def end():
            for st, _, _ in stages:
                st.readers -= 1
            for bar in after:
                bar.arrive()
        self.products.append(end)

    def run(self, roles):
        live, idle = list(roles), 0
        while live:
            moved = False
            if self.copies and self.rnd.random() < self.p_copy:
                self.copies.pop(self.rnd.randrange(len(self.copies)))()
                moved = True
            if self.products and self.rnd.random() < self.p_mma:
                self.products.pop(0)()
                moved = True
            r = self.rnd.choice(live)
            try:
                moved = next(r) or moved
            except StopIteration:
                live.remove(r)
                moved = True
            idle = 0 if moved else idle + 1
            assert idle < 20000, "no role can move"

    def leave(self):
        assert not self.copies, "a CTA ends while copies into it are in flight"
        assert not self.products, "a CTA ends while its products run"


# ---------------------------------------------------------------- single token
def decode(sequences, STAGES, PBUF, seed, broken=False, old=False):
    """`sequences`: tiles of each. Four blocks of a tile are copied one by one as their room is free."""
    sim = Sim(seed, broken)
    kfull = [Bar(1, f"KFull{s}") for s in range(STAGES)]
    kempty = [[Bar(1, f"KEmpty{s}.{k}") for k in range(4)] for s in range(STAGES)]
    sfull, pready = [Bar(1, f"SFull{i}") for i in range(2)], [Bar(2, f"PReady{i}") for i in range(2)]
    qfull, qempty, done = Bar(1, "QFull"), Bar(1, "QEmpty"), Bar(2, "Done")
    blocks = [[Stage() for _ in range(4)] for _ in range(STAGES)]
    query = Stage()
    issued = dict(it=0, sg=0, missing=0)

    def copies():
        it = sg = 0
        ok = True

        def ask():
            nonlocal sg
            qfull.arm(sg, 1)
            sim.copy(query, sg, 1, lambda: qfull.bytes(1))
            sg += 1
        for tiles in sequences:
            if not ok:
                break
            first = sg == 0
            if not first:
                ok = yield from sim.wait(qempty, sg - 1, 0)
                if not ok:
                    break
                ask()
            for _ in range(tiles):
                if first and it == STAGES:
                    ask()
                    first = False
                s, sent = it % STAGES, 0
                if it >= STAGES and not old:
                    ok = yield from sim.wait(kfull[s], it // STAGES - 1, 0)
                for k in range(4):
                    ok = ok and (it < STAGES or (yield from sim.wait(kempty[s][k], it // STAGES - 1, 0)))
                    if ok or old:       # (old: what is left of a tile goes out behind a wait that failed)
                        if k == 0:
                            kfull[s].arm(it // STAGES, 4)
                        sim.copy(blocks[s][k], it, 1, lambda s=s: kfull[s].bytes(1))
                        sent += 1
                        yield True
                it += sent > 0
                if not ok:
                    issued["missing"] = 4 - sent if sent else 0
                    break
            if ok and first:
                ask()
        issued.update(it=it, sg=sg)
        if old and not ok:
            yield from drain()

    def drain():
        if issued["missing"]:
            kfull[(issued["it"] - 1) % STAGES].bytes(issued["missing"])
        for i in range(max(0, issued["it"] - STAGES), issued["it"]):
            yield from sim.alone(kfull[i % STAGES], i // STAGES)
        if issued["sg"]:
            yield from sim.alone(qfull, issued["sg"] - 1)

    def score():
        it = 0
        ok = True
        for sg, tiles in enumerate(sequences):
            ok = ok and (yield from sim.wait(qfull, sg, 0))
            for tt in range(tiles):
                ok = ok and (it < 2 or (yield from sim.wait(pready[it & 1], (it >> 1) - 1, 0)))
                ok = ok and (yield from sim.wait(kfull[it % STAGES], it // STAGES, 0))
                if not ok:
                    break
                sim.product([(b, it, 1) for b in blocks[it % STAGES]] + [(query, sg, 1)],
                            [sfull[it & 1]] + ([qempty] if tt + 1 == tiles else []))
                it += 1
            if not ok:
                break
        sim.product([], [done])
        yield from sim.alone(done, 0)

    def value():
        it = 0
        ok = True
        for tiles in sequences:
            for _ in range(tiles):
                ok = ok and (yield from sim.wait(pready[it & 1], it >> 1, 0))
                if not ok:
                    break
                for k in range(4):
                    sim.product([(blocks[it % STAGES][k], it, 1)], [kempty[it % STAGES][k]])
                it += 1
            if not ok:
                break
        sim.product([], [done])
        yield from sim.alone(done, 0)

    def softmax():
        it = 0
        for tiles in sequences:
            for _ in range(tiles):
                yield from sim.wait(kfull[it % STAGES], it // STAGES, 0)
                yield from sim.wait(sfull[it & 1], it >> 1, 0)
                if it >= PBUF:
                    j = it - PBUF
                    yield from sim.wait(kempty[j % STAGES][3], j // STAGES, 0)
                pready[it & 1].arrive()
                yield True
                it += 1
            yield from sim.wait(kempty[(it - 1) % STAGES][3], (it - 1) // STAGES, 0)
    sim.run([copies(), score(), value(), softmax(), softmax()])
    if sim.flags[0] and not old:
        sim.run([drain()])
    sim.leave()
    return sim.expired


# ---------------------------------------------------------------- pairs of CTAs
def settle(sim, ring, mine, other, nbytes):
    n, both = len(ring), max(mine, other)
    assert both - min(mine, other) <= n
    for i in range(min(mine, other), both):
        if i >= mine:
            ring[i % n].arm(i // n, nbytes)
        else:
            ring[i % n].bytes(nbytes)
    for i in range(max(0, both - n), both):
        yield from sim.alone(ring[i % n], i // n)


def pairs_of(n, name, count=1):
    return [[Bar(count, f"{name}{s}.{r}") for r in range(2)] for s in range(n)]


def expand(units, hgs, u0, KC, STAGES, seed, broken=False, old=False):
    sim = Sim(seed, broken, 2)
    afull, bfull = [Bar(1, f"AFull{c}") for c in range(KC)], [Bar(1, f"BFull{s}") for s in range(STAGES)]
    aempty, bempty = pairs_of(KC, "AEmpty"), pairs_of(STAGES, "BEmpty")
    dfull, dempty, done = pairs_of(2, "DFull"), [Bar(2, f"DEmpty{b}") for b in range(2)], Bar(1, "Done")
    a, b = [[Stage() for _ in range(KC)] for _ in range(2)], [[Stage() for _ in range(STAGES)] for _ in range(2)]
    issued = [[0, 0], [0, 0]]

    def copies(rank):
        held, loads, it, runs, ok = -1, 0, 0, 0, True
        for u in range(u0, u0 + units):
            if not ok:
                break
            fresh = u // hgs != held
            if fresh:
                held, loads = u // hgs, loads + 1
            for c in range(KC):
                s = it % STAGES
                if fresh:
                    if ok and loads >= 2:
                        ok = yield from sim.wait(aempty[c][rank], loads - 2, rank)
                    if not ok and not old:
                        break
                    runs += 1
                    if rank == 0:
                        afull[c].arm(loads - 1, 2)
                    sim.copy(a[rank][c], loads - 1, 1, lambda c=c: afull[c].bytes(1))
                    yield True
                if ok and it >= STAGES:
                    ok = yield from sim.wait(bempty[s][rank], it // STAGES - 1, rank)
                if not ok and not old:
                    break
                if rank == 0:
                    bfull[s].arm(it // STAGES, 2)
                sim.copy(b[rank][s], it, 1, lambda s=s: bfull[s].bytes(1))
                it += 1
                yield True
        issued[rank] = [runs, it]
        if old and not ok and rank == 0:
            for c in range(KC if loads else 0):
                yield from sim.alone(afull[c], loads - 1)
            for i in range(max(0, it - STAGES), it):
                yield from sim.alone(bfull[i % STAGES], i // STAGES)

    def product():
        loads = it = 0
        ok = True
        for n in range(units):
            u = u0 + n
            fresh, last = n == 0 or u % hgs == 0, (u + 1) % hgs == 0 and n + 1 < units
            loads += fresh
            for c in range(KC):
                if fresh:
                    ok = yield from sim.wait(afull[c], loads - 1, 0)
                ok = ok and (yield from sim.wait(bfull[it % STAGES], it // STAGES, 0))
                if c == 0 and n >= 2:
                    ok = ok and (yield from sim.wait(dempty[n & 1], (n >> 1) - 1, 0))
                if not ok:
                    break
                sim.product([(a[r][c], loads - 1, 1) for r in range(2)] + [(b[r][it % STAGES], it, 1) for r in range(2)],
                            bempty[it % STAGES] + (aempty[c] if last else []))
                it += 1
            if not ok:
                break
            sim.product([], dfull[n & 1])
        sim.product([], [done])
        yield from sim.alone(done, 0)

    def out(rank):
        for n in range(units):
            if not (yield from sim.wait(dfull[n & 1][rank], n >> 1, rank)):
                break
            dempty[n & 1].arrive()
            yield True
    sim.run([copies(0), copies(1), product(), out(0), out(1)])
    if sim.flags[0] and not old:
        for ring, i in ((afull, 0), (bfull, 1)):
            sim.run([settle(sim, ring, issued[0][i], issued[1][i], 1)])
    sim.leave()
    return sim.expired


def chunk(units, NQ, STAGES, seed, broken=False, old=False, named=False, raises=0.0):
    """`units`: tiles of each."""
    sim = Sim(seed, broken, 2)
    qfull, kfull, vfull = ([Bar(1, f"{x}{s}") for s in range(n)] for x, n in (("QFull", NQ), ("KFull", STAGES), ("VFull", STAGES)))
    qempty, kempty, vempty, sfull = pairs_of(NQ, "QEmpty"), pairs_of(STAGES, "KEmpty"), pairs_of(STAGES, "VEmpty"), pairs_of(2, "SFull")
    pready, ofree, done = [Bar(2, f"PReady{g}") for g in range(2)], Bar(2, "OFree"), Bar(1, "Done")
    q, k, v = ([[Stage() for _ in range(n)] for _ in range(2)] for n in (NQ, STAGES, STAGES))
    sums = pairs_of(2, "Sums", 2)
    issued = [[0, 0, 0], [0, 0, 0]]

    def copies(rank):
        asked = keys = vals = 0
        ok = True

        def load(stages, full, n, i):
            if rank == 0:
                full[i % n].arm(i // n, 2)
            sim.copy(stages[rank][i % n], i, 1, lambda: full[i % n].bytes(1))

        def queries():
            nonlocal asked, ok
            if asked >= NQ:
                ok = yield from sim.wait(qempty[asked % NQ][rank], asked // NQ - 1, rank)
            if ok:
                load(q, qfull, NQ, asked)
                asked += 1
        for u, tiles in enumerate(units):
            if not ok:
                break
            if asked == 0:
                yield from queries()
            for j in range(tiles):
                if not ok:
                    break
                if vals >= STAGES:
                    ok = yield from sim.wait(kempty[vals % STAGES][rank], vals // STAGES - 1, rank)
                if not ok and not old:
                    break
                load(k, kfull, STAGES, keys)
                keys += 1
                yield True
                if ok and vals >= STAGES:
                    ok = yield from sim.wait(vempty[vals % STAGES][rank], vals // STAGES - 1, rank)
                if not ok and not old:
                    break
                load(v, vfull, STAGES, vals)
                vals += 1
                yield True
                if ok and j == (min(1, tiles - 1) if NQ == 2 else tiles - 1) and u + 1 < len(units):
                    yield from queries()
        issued[rank] = [asked, keys, vals]
        if old and not ok and rank == 0:
            for n, full, x in ((NQ, qfull, asked), (STAGES, kfull, keys), (STAGES, vfull, vals)):
                for i in range(max(0, x - n), x):
                    yield from sim.alone(full[i % n], i // n)

    def product():
        jt = un = last_j = 0

        def values(i, j, u):
            s = i % STAGES
            if not (yield from sim.wait(vfull[s], i // STAGES, 0)):
                return False
            if not (yield from sim.wait(pready[i & 1], i >> 1, 0)):
                return False
            if j == 0 and u > 1 and not (yield from sim.wait(ofree, u - 2, 0)):
                return False
            sim.product([(v[r][s], i, 1) for r in range(2)], vempty[s])
            return True

        def all_units():
            nonlocal jt, un, last_j
            for tiles in units:
                b, held = un % NQ, jt > 0
                if NQ == 1 and held:
                    if not (yield from values(jt - 1, last_j, un)):
                        return False
                    held = False
                if not (yield from sim.wait(qfull[b], un // NQ, 0)):
                    return False
                un += 1
                for j in range(tiles):
                    s = jt % STAGES
                    if not (yield from sim.wait(kfull[s], jt // STAGES, 0)):
                        return False
                    sim.product([(k[r][s], jt, 1) for r in range(2)] + [(q[r][b], un - 1, 1) for r in range(2)],
                                kempty[s] + sfull[jt & 1] + (qempty[b] if j + 1 == tiles else []))
                    if held and not (yield from values(jt - 1, last_j, un if j else un - 1)):
                        return False
                    held, last_j, jt = True, j, jt + 1
            return True
        ok = yield from all_units()
        if ok and jt:
            yield from values(jt - 1, last_j, un)
        sim.product([], [done])
        yield from sim.alone(done, 0)

    def softmax(rank, g):
        jt = 0
        for un, tiles in enumerate(units):
            off = (jt & 1) ^ g
            for i, j in enumerate(range(jt + off, jt + tiles, 2)):
                yield from sim.wait(sfull[g][rank], j >> 1, rank)
                if i and sim.rnd.random() < raises:
                    yield from sim.wait(vempty[(j - 2) % STAGES][rank], (j - 2) // STAGES, rank)
                pready[g].arrive()
                yield True
            left = sums[un & 1][rank]
            at = left.phase
            left.arrive()
            yield True
            if g == (jt + tiles - 1) & 1:
                if named:       # a named barrier: no limit, and whoever arrives counts
                    while left.phase == at:
                        yield False
                else:
                    yield from sim.wait(left, un >> 1, rank)
                for j in range(max(jt, jt + tiles - 2), jt + tiles):
                    yield from sim.wait(vempty[j % STAGES][rank], j // STAGES, rank)
                ofree.arrive()
                yield True
            jt += tiles
    sim.run([copies(0), copies(1), product()] + [softmax(r, g) for r in range(2) for g in range(2)])
    if sim.flags[0] and not old:
        for i, ring in enumerate((qfull, kfull, vfull)):
            sim.run([settle(sim, ring, issued[0][i], issued[1][i], 1)])
    sim.leave()
    return sim.expired


DECODE = [((1,), 2, 2), ((3, 1, 2), 2, 1), ((7,), 2, 2), ((1, 1, 1, 1, 5), 4, 2), ((9, 4), 4, 2)]
EXPAND = [(1, 4, 0, 8, 5), (5, 3, 0, 8, 5), (6, 2, 1, 8, 5), (4, 1, 0, 8, 5), (7, 3, 2, 4, 8)]
CHUNK = [((1,), 2, 3), ((2, 2, 2), 2, 3), ((1, 1, 1, 1), 2, 4), ((9, 5, 3), 2, 3), ((8,), 1, 4), ((4, 1, 3, 6), 1, 4), ((3, 2, 1, 2, 3), 1, 4)]
KERNELS = [(decode, c) for c in DECODE] + [(expand, c) for c in EXPAND] + [(chunk, c) for c in CHUNK]
IDS = [f"{f.__name__} {' '.join(map(str, c))}" for f, c in KERNELS]


@pytest.mark.parametrize("kernel,sizes", KERNELS, ids=IDS)
def test_whole_runs(kernel, sizes):
    for seed in range(12):
        assert kernel(*sizes, seed, **({"raises": 0.5} if kernel is chunk and seed % 2 else {})) == 0


@pytest.mark.parametrize("kernel,sizes", KERNELS, ids=IDS)
def test_a_wait_that_runs_out_leaves_nothing_behind(kernel, sizes):
    assert sum(kernel(*sizes, seed, broken=True) for seed in range(60)) > 0


@pytest.mark.parametrize("kernel,sizes", [(decode, DECODE), (expand, EXPAND), (chunk, CHUNK)], ids=["decode", "expand", "chunk"])
def test_model_sees_copies_behind_a_failed_wait(kernel, sizes):
    """Arming and copying on behind a wait that failed, and waiting for the copies only where the copying warp itself gave up."""
    seen = set()
    for seed in range(40):
        for some in sizes:
            try:
                kernel(*some, seed, broken=True, old=True)
            except AssertionError as e:
                seen |= {m for m in ("armed for phase", "over a stage", "in flight") if m in str(e)}
    assert "armed for phase" in seen and "in flight" in seen, seen


def test_model_sees_a_named_barrier_behind_a_failed_wait():
    """The half of the softmax that only arrives runs ahead once no wait holds it, completes the other's barrier by itself, and the
    other's last wait, which has no limit, never ends."""
    stuck = 0
    for seed in range(40):
        for some in CHUNK:
            try:
                chunk(*some, seed, broken=True, named=True)
            except AssertionError as e:
                assert "no role can move" in str(e)
                stuck += 1
        assert chunk(*CHUNK[3], seed, named=True) == 0
    assert stuck
