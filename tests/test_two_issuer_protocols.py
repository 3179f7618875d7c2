"""Model check of the barrier protocols with two threads that issue products (no GPU): the tiled FP8_B128 product
(stages in pairs) and the few-token layer (two sets of epilogue warps that take units in turn, a result slot per
stage or per unit).  The model is test_barrier_protocols': the kernels' own counts, counters and parities, copies
that land in any order, tensor work that completes in the order of the thread that issued it."""
import pytest

from test_barrier_protocols import Bar, Sim, Violation, check


class Ring:
    """The TMA ring: full (count, with `loads` copies per stage) and empty."""

    def __init__(self, sim, NS, loads=1):
        self.sim, self.NS, self.loads = sim, NS, loads
        self.full, self.empty = [Bar(loads) for _ in range(NS)], [Bar(1) for _ in range(NS)]
        self.tag, self.fresh = [None] * NS, [0] * NS

    def land(self, s, tag):
        def copied():
            check(self.fresh[s] == 0 or self.tag[s] == tag, f"stage {s} was overwritten before it was used")
            self.tag[s] = tag
            self.fresh[s] += 1
            self.full[s].arrive()
        self.sim.post(None, copied)

    def producer(self, units, enter=None):
        n = 0
        for u, k_stages in enumerate(units):
            if enter:
                yield from enter(u)
            for ks in range(k_stages):
                s, ph = n % self.NS, n // self.NS & 1
                yield lambda s=s, ph=ph: self.empty[s].passed(ph ^ 1)
                self.land(s, (u, ks))
                n += 1

    def wait(self, n):
        s, ph = n % self.NS, n // self.NS & 1
        yield lambda: self.full[s].passed(ph)

    def use(self, n, tag, m, done):
        """Products of stage n by issuer m; done(): what completes with them."""
        s = n % self.NS
        check(self.tag[s] == tag and self.fresh[s] == self.loads, f"products of {self.tag[s]}, expected {tag}")

        def finished():
            self.fresh[s] = 0
            done()
            self.empty[s].arrive()
        self.sim.post(("tc", m), finished)


def mine(n, ks, m, NS, plant):
    """Whether a stage is issuer m's: by the ring's slot, so that a slot's uses are all one issuer's.  (By turns
    within a unit, the parity of full could be that of the use two back.)"""
    return (ks if plant == "by_turns" else n % NS) % 2 == m


def pairs(sim, units, NS, n_epi=8, plant=None):
    """linear_tile_kernel: two pair slots, a tile's stages in pairs."""
    ring = Ring(sim, NS)
    pfull, pempty = [Bar(2) for _ in range(2)], [Bar(n_epi) for _ in range(2)]
    part, readers = [[None, None], [None, None]], [[n_epi, n_epi], [n_epi, n_epi]]

    def mma(m):
        n, ps, pph = 0, 0, 0
        for u, k_stages in enumerate(units):
            for ks in range(k_stages):
                last = ks == k_stages - 1
                if mine(n, ks, m, NS, plant):
                    yield from ring.wait(n)
                    yield lambda ps=ps, pph=pph: pempty[ps].passed(pph ^ 1)
                    check(readers[ps][ks % 2] == n_epi, "a product was overwritten before it was read")

                    def done(ps=ps, tag=(u, ks)):
                        part[ps][tag[1] % 2], readers[ps][tag[1] % 2] = tag, 0
                        pfull[ps].arrive()
                    ring.use(n, (u, ks), m, done)
                elif last and ks % 2 == 0:
                    if plant != "eager":
                        yield lambda ps=ps, pph=pph: pempty[ps].passed(pph ^ 1)
                    pfull[ps].arrive()
                n += 1
                if ks % 2 == 1 or last:
                    ps, pph = (ps + 1) % 2, pph ^ (ps == 1)

    def epilogue():
        ps, pph = 0, 0
        for u, k_stages in enumerate(units):
            for ks in range(0, k_stages, 2):
                yield lambda ps=ps, pph=pph: pfull[ps].passed(pph)
                for sub in range(2 if ks + 1 < k_stages else 1):
                    check(part[ps][sub] == (u, ks + sub), f"sums of {part[ps][sub]}, expected {(u, ks + sub)}")
                    readers[ps][sub] += 1
                    yield lambda: True
                pempty[ps].arrive()
                ps, pph = (ps + 1) % 2, pph ^ (ps == 1)

    sim.role("producer", ring.producer(units))
    for m in range(2):
        sim.role(f"mma{m}", mma(m))
    for w in range(n_epi):
        sim.role(f"epilogue{w}", epilogue())


def few(sim, units, NS, block, n_epi=4, plant=None):
    """few_layer_kernel on one CTA: weights and columns by threads of their own, two issuers, two sets of epilogue
    warps with slots of their own (8 each, one per stage, or one each, per unit)."""
    ring = Ring(sim, NS, loads=2)
    slots = 8 if block else 1
    rfull = [Bar(1 if block else 2) for _ in range(2 * slots)]
    rempty = [Bar(n_epi) for _ in range(2 * slots)]
    UQ = 4
    uq_full, uq_empty = [Bar(1) for _ in range(UQ)], [Bar(1 + 2 + 2 * n_epi) for _ in range(UQ)]
    part, readers = [None] * (2 * slots), [n_epi] * (2 * slots)

    def publish(u):
        yield lambda: uq_empty[u % UQ].passed(u // UQ & 1 ^ 1)
        uq_full[u % UQ].arrive()

    def next_unit(u):
        yield lambda: uq_full[u % UQ].passed(u // UQ & 1)
        uq_empty[u % UQ].arrive()

    def mma(m):
        n, slot, other, sph, oph, end = 0, 0, slots, 0, 0, slots
        for u, k_stages in enumerate(units):
            yield from next_unit(u)
            if not block:
                yield lambda slot=slot, sph=sph: rempty[slot].passed(sph ^ 1)
                check(readers[slot] == n_epi or part[slot] == (u, None), "a sum was overwritten before it was read")
            for ks in range(k_stages):
                if mine(n, ks, m, NS, plant):
                    yield from ring.wait(n)
                    if block:
                        yield lambda slot=slot, sph=sph: rempty[slot].passed(sph ^ 1)
                        check(readers[slot] == n_epi, "a product was overwritten before it was read")

                    def done(slot=slot, tag=(u, ks)):
                        if block:
                            part[slot], readers[slot] = tag, 0
                            rfull[slot].arrive()
                    ring.use(n, (u, ks), m, done)
                n += 1
                if block or ks == k_stages - 1:
                    if not block:
                        def unit_done(slot=slot, u=u):
                            part[slot] = (u, None)
                            readers[slot] = 0
                            rfull[slot].arrive()
                        sim.post(("tc", m), unit_done)
                    slot += 1
                    if slot == end:
                        slot, sph = end - slots, sph ^ 1
            if plant == "one_set":
                continue
            slot, other, sph, oph, end = other, slot, oph, sph, 3 * slots - end

    def epilogue(st):
        slot, sph = st * slots, 0
        for u, k_stages in enumerate(units):
            yield from next_unit(u)
            if u % 2 != st:
                continue
            for ks in range(k_stages) if block else [None]:
                yield lambda slot=slot, sph=sph: rfull[slot].passed(sph)
                check(part[slot] == (u, ks), f"sums of {part[slot]}, expected {(u, ks)}")
                readers[slot] += 1
                rempty[slot].arrive()
                slot += 1
                if slot == (st + 1) * slots:
                    slot, sph = st * slots, sph ^ 1
                yield lambda: True

    sim.role("weights", ring.producer(units, publish))
    sim.role("columns", ring.producer(units, next_unit))
    for m in range(2):
        sim.role(f"mma{m}", mma(m))
    for w in range(2 * n_epi):
        sim.role(f"epilogue{w}", epilogue(w // n_epi))


UNITS = [[1], [1, 1, 1, 1, 1], [2, 2, 2], [3, 3, 3, 3], [5, 5, 5, 5], [21, 21, 21], [9, 9, 9, 1, 1, 1, 1, 1, 1, 1, 1],
         [1] * 20 + [3] * 7, [1] * 17 + [2] * 9, [8, 8, 8, 15, 15]]


@pytest.mark.parametrize("units", UNITS)
@pytest.mark.parametrize("NS", [2, 4, 6, 8])
def test_tiled_product_protocol(units, NS):
    units = [units[0]] * len(units)   # a product's tiles have one number of stages
    for seed in range(10):
        sim = Sim(seed)
        pairs(sim, units, NS, n_epi=3)
        assert sim.run() == "done"


@pytest.mark.parametrize("units", UNITS)
@pytest.mark.parametrize("NS", [2, 8, 10, 12])
@pytest.mark.parametrize("block", [False, True])
def test_few_token_layer_protocol(units, NS, block):
    for seed in range(10):
        sim = Sim(seed)
        few(sim, units, NS, block, n_epi=2)
        assert sim.run() == "done"


def caught(build, seeds=40):
    for seed in range(seeds):
        sim = Sim(seed)
        try:
            build(sim)
            if sim.run(200_000) != "done":
                return True
        except (Violation, AssertionError):
            return True
    return False


def test_planted_mistakes_are_caught():
    assert caught(lambda sim: pairs(sim, [3, 3, 3, 3, 3], 4, n_epi=3, plant="eager"))
    assert caught(lambda sim: few(sim, [5, 5, 5, 5], 4, True, n_epi=2, plant="one_set"))
    assert caught(lambda sim: pairs(sim, [3] * 8, 2, n_epi=3, plant="by_turns"), 400)
    assert caught(lambda sim: few(sim, [3] * 8, 2, False, n_epi=2, plant="by_turns"), 400)
