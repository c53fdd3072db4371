"""Model check of the barriers between the warps of the attention kernel for
chunks, on the CPU.

Two loading warps (K and V) fill a ring of shared-memory stages; a product
warp per query tile issues S_i = Q_i K^T and O_i += P_i V, the two taking
turns; the softmax warps of a tile turn S into the weights P, in place.  The
model replays this under random interleavings: no step takes any particular
time, copies land in any order, and products run after they were issued, in
the order of their own thread alone.  Barriers only show phase parity, as on
the card (``Bar`` of test_pipeline_protocol).

Checked: nothing stalls, every product finds the tile, the queries and the
weights that it is meant for (when it runs, not when it is issued), and no
copy lands in a stage that a product still reads.
"""

import random

import pytest

from test_pipeline_protocol import Bar

WARPS = 2        # softmax warps of a query tile (four on the card)


class Wrong(AssertionError):
    pass


class Stall(AssertionError):
    pass


class GaveUp(Exception):
    pass


class Machine:
    """Actors are generators that yield (barrier, parity) to wait, or None
    between two steps.  Tensor-core queues and copies in flight act too.
    gives_up: an actor and which of its waits runs out at once (not one for
    its own copies or products, which do end); every other wait then runs out
    where nothing moves any more."""

    def __init__(self, seed, gives_up=None):
        self.rnd = random.Random(seed)
        self.actors, self.waits = {}, {}
        self.flying, self.queues = [], {}
        self.gives_up, self.waited, self.gave_up = gives_up, {}, 0

    def add(self, name, gen):
        self.actors[name], self.waits[name] = gen, None

    def step(self, a, gone=False):
        self.gave_up += gone
        try:
            w = self.actors[a].throw(GaveUp()) if gone else next(self.actors[a])
            if w is not None and len(w) == 2 and self.gives_up and self.gives_up[0] == a:
                self.waited[a] = self.waited.get(a, 0) + 1
                if self.waited[a] == self.gives_up[1]:
                    return self.step(a, gone=True)
            self.waits[a] = w
        except StopIteration:
            del self.actors[a], self.waits[a]
            if not self.actors and (self.flying or any(self.queues.values())):
                raise Wrong("copies or products are left behind")

    def run(self, most=200000):
        rnd, idle = self.rnd, 0
        # some interleavings hold one actor back for long
        slow = rnd.choice([None, *self.actors, *self.queues, "copies"])
        for _ in range(most):
            ready = [*self.actors] + [q for q in self.queues if self.queues[q]] + \
                    (["copies"] if self.flying else [])
            if not ready:
                return
            a = rnd.choice(ready)
            if a == slow and idle < 40 and rnd.random() < 0.97:
                idle += 1
                continue
            if a == "copies":
                self.flying.pop(rnd.randrange(len(self.flying)))()
            elif a in self.queues:
                self.queues[a].pop(0)()
            else:
                w = self.waits[a]
                if w is not None and not w[0].try_wait(w[1] & 1):
                    idle += 1
                    if idle > 60 * len(ready) and not self.flying and \
                            not any(self.queues.values()) and \
                            not any(w is None or w[0].try_wait(w[1] & 1)
                                    for w in self.waits.values()):
                        if not self.gave_up:
                            raise Stall(sorted(self.actors))
                        self.step(a, gone=True)
                    continue
                self.step(a)
            idle = 0
        raise Stall("no end")


def ending(body, end, always):
    """A role: its body until that ends or a wait runs out, then its end
    (whose waits may run out too), always or after a wait of its own."""
    gone = not always
    try:
        yield from body
    except GaveUp:
        gone = False
    if gone:
        return
    for w in end():
        try:
            yield (*w, "end")
        except GaveUp:
            pass


def chunk(seed, units, stages, hand_back=True, one_queue=False, both_release=True,
          step_along=True, in_order=True, gives_up=None, ends=True):
    """units of one CTA: (query tiles, token tiles, set of token tiles whose V
    the loading warp mends).  one_queue: the products of both threads run in
    the order in which they were issued.  both_release: a stage is free once
    both product warps have let it go, the second one in units of one query
    tile too, after the stage's copy (step_along) or ahead of it."""
    m = Machine(seed)
    NS = stages
    full = [Bar(1) for _ in range(NS)]
    empty = [Bar(2 if both_release else 1) for _ in range(NS)]
    q_full, p_half, p_ready = ([Bar(WARPS), Bar(WARPS)] for _ in range(3))
    s_full, o_full, turns = ([Bar(1), Bar(1)] for _ in range(3))
    fix, loaded, released = Bar(1), Bar(1), Bar(2 * WARPS)
    ring = [None] * NS
    queries, s_at, o_at = [None, None], [None, None], [None, None]
    p_at = [[None, None] for _ in range(2)]
    at, drain = [0, 1], [Bar(1), Bar(1)]
    out = {}

    def expect(got, want):
        if got != want:
            raise Wrong(f"{got} where {want} is meant")

    def load(half):
        it, n_fix = half, 0
        for n, (tiles, nk, mends) in enumerate(units):
            for k in range(nk):
                s = it % NS
                if it >= NS:
                    yield empty[s], it // NS - 1
                mend = half == 1 and k in mends
                bar, tag = fix if mend else full[s], (n, half, k)
                ring[s] = None
                bar.arrive(tx=1)

                def land(s=s, bar=bar, tag=tag):
                    ring[s] = tag
                    bar.land(1)
                m.flying.append(land)
                at[half] = it + 2
                yield None
                if mend:
                    yield fix, n_fix
                    n_fix += 1
                    expect(ring[s], tag)
                    full[s].arrive()
                it += 2
                at[half] = it
            if half:
                if n > 0:
                    yield released, n - 1
                loaded.arrive()

    def products(i):
        q = m.queues["T0" if one_queue else f"T{i}"]
        it = n_q = n_p = n_t = steps = 0

        def product_s(s, n, k):
            def run():
                expect(ring[s], (n, 0, k))
                expect(queries[i], [n] * WARPS)
                s_at[i], p_at[i] = (n, k), [None, None]
            return run

        def product_o(s, n, k, part):
            def run():
                expect(ring[s], (n, 1, k))
                expect(p_at[i][part], [(n, k)] * WARPS)
                o_at[i] = (n, k, part)
            return run
        for n, (tiles, nk, _) in enumerate(units):
            if i >= tiles:
                for it in range(it, it + 2 * nk):
                    if both_release:
                        if step_along:
                            yield full[it % NS], it // NS
                        if in_order:
                            q.append(empty[it % NS].arrive)
                        else:
                            empty[it % NS].arrive()
                it += 1 if nk else 0
                continue
            lets_go, pair = both_release or i == tiles - 1, tiles == 2
            for k in range(nk + 1 if nk else 0):
                do_o, do_s = k > 0, k < nk
                vs = it % NS
                if do_o:
                    yield full[vs], it // NS
                    it += 1
                ks = it % NS
                if do_s:
                    yield full[ks], it // NS
                    it += 1
                    if k == 0:
                        yield q_full[i], n_q
                        n_q += 1
                if do_o:
                    yield p_half[i], n_p
                if pair and (i == 1 or (steps > 0 if hand_back else k > 0)):
                    yield turns[i], n_t
                    n_t += 1
                if do_o:
                    q.append(product_o(vs, n, k - 1, 0))
                    yield p_ready[i], n_p
                    n_p += 1
                    q.append(product_o(vs, n, k - 1, 1))
                    if not do_s:
                        q.append(o_full[i].arrive)
                    if lets_go:
                        q.append(empty[vs].arrive)
                if do_s:
                    q.append(product_s(ks, n, k))
                    q.append(s_full[i].arrive)
                    if lets_go:
                        q.append(empty[ks].arrive)
                if pair:
                    if hand_back or i == 0 or do_s:
                        turns[1 - i].arrive()
                    steps += 1
                yield None

    def softmax(i, w):
        n_s = n_o = 0
        for n, (tiles, nk, _) in enumerate(units):
            if i < tiles and nk > 0:
                if queries[i] is None:
                    queries[i] = [None] * WARPS
                queries[i][w] = n
                q_full[i].arrive()
                for k in range(nk):
                    yield s_full[i], n_s
                    n_s += 1
                    expect(s_at[i], (n, k))
                    yield None
                    for part, bar in ((0, p_half[i]), (1, p_ready[i])):
                        if p_at[i][part] is None:
                            p_at[i][part] = [None] * WARPS
                        p_at[i][part][w] = (n, k)
                        bar.arrive()
                        yield None
                yield o_full[i], n_o
                n_o += 1
                expect(o_at[i], (n, nk - 1, 1))
            yield loaded, n
            if i < tiles:
                out[n, i, w] = True
            released.arrive()

    def landed(half):
        first = max(0, at[half] - NS)
        return [(full[it % NS], it // NS) for it in range(first, at[half]) if it % 2 == half]

    def drained(i):
        m.queues["T0" if one_queue else f"T{i}"].append(drain[i].arrive)
        return [(drain[i], 0)]

    for half in (0, 1):
        m.add(f"load{half}", ending(load(half), lambda half=half: landed(half), ends))
    for i in (0, 1):
        m.queues[f"T{i}"] = []
        m.add(f"products{i}", ending(products(i), lambda i=i: drained(i), ends))
        for w in range(WARPS):
            m.add(f"softmax{i}.{w}", ending(softmax(i, w), list, ends))
    m.run()
    assert gives_up or len(out) == sum(t for t, _, _ in units) * WARPS


def random_units(rnd, pairs_only=False):
    units = []
    for _ in range(rnd.randint(1, 5)):
        nk = rnd.choice([0, 1, 1, 2, 3, 4, 7])
        units.append((2 if pairs_only else rnd.choice([1, 2, 2]), nk,
                      {k for k in range(nk) if rnd.random() < 0.3}))
    return units


def fails(what, trials, **kw):
    """The trials' first failure of a kind, or None."""
    for trial in range(trials):
        rnd = random.Random(trial)
        try:
            chunk(trial, random_units(rnd, kw.get("pairs_only", False)), rnd.choice([5, 10]),
                  **{k: v for k, v in kw.items() if k != "pairs_only"})
        except what as e:
            return trial, e
    return None


def test_turns_of_the_query_tiles_never_stall():
    """Every unit ends, whichever tile is late (the rule: each step is handed
    over, a unit's last one too, and waited for)."""
    assert fails((Stall, Wrong), 1500, one_queue=True, pairs_only=True) is None


def test_model_catches_a_last_step_that_is_not_handed_over():
    """Without it tile 0 may hand over twice before tile 1 has looked: the
    parity then reads as if it had not, and both wait for good."""
    assert fails(Stall, 1500, one_queue=True, pairs_only=True, hand_back=False) is not None


def test_stages_are_free_when_both_tiles_products_have_read_them():
    """Products of the two threads run in any order among each other, and
    units of one and two query tiles follow one another."""
    assert fails((Stall, Wrong), 3000) is None


def test_model_catches_a_release_by_the_last_tile_alone():
    """A commit speaks for its own thread's products: tile 0's may still read
    the stage.  And where a unit of one tile follows one of two, tile 0 may
    let its stages go before tile 1 has let go of the unit before, so that a
    loading warp takes one release for another."""
    assert fails(Wrong, 1500, both_release=False, pairs_only=True) is not None
    assert fails((Stall, Wrong), 1500, both_release=False, one_queue=True) is not None


def test_model_catches_releases_out_of_order():
    """The warp without rows lets go of a stage once its copy is there, and
    behind its own products: ahead of the copy the release would count for the
    stage's use before, and ahead of the products a later stage would be free
    before an earlier one, where a loading warp looks at every other use of a
    stage only."""
    assert fails((Stall, Wrong), 3000, step_along=False) is not None
    assert fails((Stall, Wrong), 3000, in_order=False) is not None


def leavings(trials, **kw):
    for trial in range(trials):
        rnd = random.Random(trial)
        units, stages = random_units(rnd), rnd.choice([5, 10])
        name = rnd.choice(["load0", "load1", "products0", "products1", "softmax0.0", "softmax1.1"])
        try:
            chunk(trial, units, stages, gives_up=(name, rnd.randint(1, 12)), **kw)
        except (Stall, Wrong) as e:
            return trial, e
    return None


def test_nothing_is_left_behind_when_a_wait_runs_out():
    """Copies and products that were issued end before the CTA does, whichever
    role's wait ran out."""
    assert leavings(1500) is None


def test_model_catches_roles_that_leave_their_work_behind():
    assert leavings(1500, ends=False) is not None


def test_nothing_is_left_behind_whichever_wait_runs_out(monkeypatch):
    """As above, with the machine told of the wait (``chunk`` makes its machine
    without)."""
    gave = 0
    for trial in range(1500):
        rnd = random.Random(trial)
        units, stages = random_units(rnd), rnd.choice([5, 10])
        who = rnd.choice(["load0", "load1", "products0", "products1", "softmax0.0", "softmax1.1"])
        machine = Machine(trial, (who, rnd.randint(1, 12)))
        with monkeypatch.context() as m:
            m.setattr(f"{__name__}.Machine", lambda seed, machine=machine: machine)
            chunk(trial, units, stages, gives_up=machine.gives_up)
        gave += machine.gave_up > 0
    assert gave > 750


# ---------------------------------------------------------------------------
# Chunks over caches of bytes
# ---------------------------------------------------------------------------

CONVERT = 2      # converting warps (four on the card)


def over_bytes(seed, units, stages, places=None, both_scales=True, all_loaded=True,
               wait_released=True, gives_up=None, ends=True):
    """As chunk, over a cache of bytes: no copies, but converting warps that
    each write their part of a stage, and of the scales of its tile; what they
    take out of a unit they note, twice over.  units: (query tiles, token tiles).
    places: tiles whose scales have room, the stages' number by default.
    both_scales: a tile's scales are there when K's and V's have come.  all_loaded:
    a unit is loaded when every warp says so.  wait_released: the warps keep one
    unit ahead of the softmax at most."""
    m = Machine(seed, gives_up)
    NS, NP = stages, places or stages
    full, empty = [Bar(CONVERT) for _ in range(NS)], [Bar(2) for _ in range(NS)]
    q_full, p_half, p_ready = ([Bar(WARPS), Bar(WARPS)] for _ in range(3))
    s_full, o_full, turns = ([Bar(1), Bar(1)] for _ in range(3))
    scales = [Bar((2 if both_scales else 1) * CONVERT) for _ in range(NP)]
    loaded, released = Bar(CONVERT if all_loaded else 1), Bar(2 * WARPS)
    ring = [[None] * CONVERT for _ in range(NS)]
    scale_at = [[[None] * CONVERT for _ in range(2)] for _ in range(NP)]
    notes = [[None] * CONVERT for _ in range(2)]
    queries, s_at, o_at = [None, None], [None, None], [None, None]
    p_at = [[None, None] for _ in range(2)]
    drain, out = [Bar(1), Bar(1)], {}

    def expect(got, want):
        if got != want:
            raise Wrong(f"{got} where {want} is meant")

    def convert(w):
        tile = 0
        for n, (_, nk) in enumerate(units):
            for k in range(nk):
                for half in (0, 1):
                    s, turn = (2 * tile + half) % NS, (2 * tile + half) // NS
                    if turn > 0:
                        yield empty[s], turn - 1
                    scale_at[tile % NP][half][w] = (n, k)
                    yield None
                    ring[s][w] = (n, half, k)
                    yield None
                    if both_scales or half == 0:
                        scales[tile % NP].arrive()
                    full[s].arrive()
                    yield None
                notes[n & 1][w] = n
                tile += 1
            notes[n & 1][w] = n
            if n > 0 and wait_released:
                yield released, n - 1
            if all_loaded or w == 0:
                loaded.arrive()
            yield None

    def products(i):
        q = m.queues[f"T{i}"]
        it = n_q = n_p = n_t = steps = 0

        def product_s(s, n, k):
            def run():
                expect(ring[s], [(n, 0, k)] * CONVERT)
                expect(queries[i], [n] * WARPS)
                s_at[i], p_at[i] = (n, k), [None, None]
            return run

        def product_o(s, n, k, part):
            def run():
                expect(ring[s], [(n, 1, k)] * CONVERT)
                expect(p_at[i][part], [(n, k)] * WARPS)
                o_at[i] = (n, k, part)
            return run
        for n, (tiles, nk) in enumerate(units):
            if i >= tiles:
                for _ in range(2 * nk):
                    yield full[it % NS], it // NS
                    q.append(empty[it % NS].arrive)
                    it += 1
                continue
            for k in range(nk + 1 if nk else 0):
                do_o, do_s = k > 0, k < nk
                vs = it % NS
                if do_o:
                    yield full[vs], it // NS
                    it += 1
                ks = it % NS
                if do_s:
                    yield full[ks], it // NS
                    it += 1
                    if k == 0:
                        yield q_full[i], n_q
                        n_q += 1
                if do_o:
                    yield p_half[i], n_p
                if tiles == 2 and (i == 1 or steps > 0):
                    yield turns[i], n_t
                    n_t += 1
                if do_o:
                    q.append(product_o(vs, n, k - 1, 0))
                    yield p_ready[i], n_p
                    n_p += 1
                    q.append(product_o(vs, n, k - 1, 1))
                    if not do_s:
                        q.append(o_full[i].arrive)
                    q.append(empty[vs].arrive)
                if do_s:
                    q.append(product_s(ks, n, k))
                    q.append(s_full[i].arrive)
                    q.append(empty[ks].arrive)
                if tiles == 2:
                    turns[1 - i].arrive()
                    steps += 1
                yield None

    def softmax(i, w):
        n_s = n_o = tile0 = 0
        for n, (tiles, nk) in enumerate(units):
            if i < tiles and nk > 0:
                if queries[i] is None:
                    queries[i] = [None] * WARPS
                queries[i][w] = n
                q_full[i].arrive()
                for k in range(nk):
                    yield s_full[i], n_s
                    n_s += 1
                    t = tile0 + k
                    yield scales[t % NP], t // NP
                    expect(scale_at[t % NP][0], [(n, k)] * CONVERT)    # for the maximum
                    yield None
                    for part, bar in ((0, p_half[i]), (1, p_ready[i])):
                        expect(s_at[i], (n, k))
                        expect(scale_at[t % NP], [[(n, k)] * CONVERT] * 2)
                        if p_at[i][part] is None:
                            p_at[i][part] = [None] * WARPS
                        p_at[i][part][w] = (n, k)
                        bar.arrive()
                        yield None
                yield o_full[i], n_o
                n_o += 1
                expect(o_at[i], (n, nk - 1, 1))
            yield loaded, n
            expect(notes[n & 1], [n] * CONVERT)
            yield None
            expect(notes[n & 1], [n] * CONVERT)
            if i < tiles:
                out[n, i, w] = True
            tile0 += nk
            released.arrive()

    def drained(i):
        m.queues[f"T{i}"].append(drain[i].arrive)
        return [(drain[i], 0)]

    for w in range(CONVERT):
        m.add(f"convert{w}", ending(convert(w), list, ends))
    for i in (0, 1):
        m.queues[f"T{i}"] = []
        m.add(f"products{i}", ending(products(i), lambda i=i: drained(i), ends))
        for w in range(WARPS):
            m.add(f"softmax{i}.{w}", ending(softmax(i, w), list, ends))
    m.run()
    assert gives_up or len(out) == sum(t for t, _ in units) * WARPS


def over_bytes_fails(what, trials, gives_up=False, **kw):
    for trial in range(trials):
        rnd = random.Random(trial)
        units = [(rnd.choice([1, 2, 2]), rnd.choice([0, 1, 1, 2, 3, 4, 7]))
                 for _ in range(rnd.randint(1, 6))]
        who = rnd.choice(["convert0", "convert1", "products0", "products1", "softmax0.0", "softmax1.1"])
        try:
            over_bytes(trial, units, rnd.choice([4, 8]),
                       gives_up=(who, rnd.randint(1, 12)) if gives_up else None, **kw)
        except what as e:
            return trial, e
    return None


def test_bytes_reach_the_products_as_the_tiles_they_are_meant_for():
    """Stages, scales and notes, under any order of the converting warps."""
    assert over_bytes_fails((Stall, Wrong), 2000) is None


def test_model_catches_scales_that_are_overwritten_or_early():
    """With room for one tile's scales the next tile's come while the softmax
    reads; and K's scales alone do not say that V's are there."""
    assert over_bytes_fails(Wrong, 2000, places=1) is not None
    assert over_bytes_fails(Wrong, 2000, both_scales=False) is not None


def test_model_catches_notes_that_are_read_early_or_overwritten():
    """One converting warp's word does not go for the others', and without the
    wait for the softmax its notes of two units before are lost (or a unit's
    phase passes for the one before)."""
    assert over_bytes_fails(Wrong, 2000, all_loaded=False) is not None
    assert over_bytes_fails((Stall, Wrong), 2000, wait_released=False) is not None


def test_bytes_leave_no_products_behind_when_a_wait_runs_out():
    assert over_bytes_fails((Stall, Wrong), 1500, gives_up=True) is None
    assert over_bytes_fails((Stall, Wrong), 1500, gives_up=True, ends=False) is not None


# ---------------------------------------------------------------------------
# Attention mass of many rows
# ---------------------------------------------------------------------------

def mass(seed, units, watch_all=True, gives_up=None, ends=True):
    """The mass kernel: a warp loads a unit's K tiles (four slots) and the
    query tiles that pass by (three), a warp reads the log-sum-exps of their
    rows (three), a product warp per K tile writes S to two buffers in turn,
    and the sums of a tile are made in two halves.  units: (K tiles, query
    tiles).  watch_all: a product warp waits for both K tiles of a unit, and
    lets the one that it does not read go at once.  ends: as in chunk."""
    m = Machine(seed, gives_up)
    k_full, k_empty = ([Bar(1) for _ in range(4)], [Bar(2 if watch_all else 1) for _ in range(4)])
    q_full, q_empty = [Bar(1) for _ in range(3)], [Bar(2) for _ in range(3)]
    l_full, l_empty = [Bar(1) for _ in range(3)], [Bar(4) for _ in range(3)]
    s_full = [[Bar(1), Bar(1)] for _ in range(2)]
    s_empty = [[Bar(2), Bar(2)] for _ in range(2)]
    half_done, half_free = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    keys, queries, lses = [None] * 4, [None] * 3, [None] * 3
    s_at, half_at, out = [[None, None], [None, None]], [None, None], {}
    at, drain = [0, 0], [Bar(1), Bar(1)]

    def expect(got, want):
        if got != want:
            raise Wrong(f"{got} where {want} is meant")

    def copy(room, slot, tag, bar):
        def land():
            room[slot] = tag
            bar.land(1)
        room[slot] = None
        bar.arrive(tx=1)
        m.flying.append(land)

    def loads():
        n_k = n_q = 0
        for n, (tiles, steps) in enumerate(units):
            if steps == 0:
                continue
            for i in range(tiles):
                if n_k >= 4:
                    yield k_empty[n_k % 4], n_k // 4 - 1
                copy(keys, n_k % 4, (n, i), k_full[n_k % 4])
                n_k += 1
                at[0] = n_k
                yield None
            for t in range(steps):
                if n_q >= 3:
                    yield q_empty[n_q % 3], n_q // 3 - 1
                copy(queries, n_q % 3, (n, t), q_full[n_q % 3])
                n_q += 1
                at[1] = n_q
                yield None

    def rows():
        n_l = 0
        for n, (_, steps) in enumerate(units):
            for t in range(steps):
                if n_l >= 3:
                    yield l_empty[n_l % 3], n_l // 3 - 1
                lses[n_l % 3] = (n, t)
                l_full[n_l % 3].arrive()
                n_l += 1
                yield None

    def products(i):
        q = m.queues[f"T{i}"]
        n_k = n_s = n_l = 0

        def product(k_slot, q_slot, buf, n, t):
            def run():
                expect(keys[k_slot], (n, i))
                expect(queries[q_slot], (n, t))
                s_at[i][buf] = (n, t)
            return run
        for n, (tiles, steps) in enumerate(units):
            if steps == 0:
                continue
            work = i < tiles
            k_slot = (n_k + i) % 4
            for j in range(tiles):
                if watch_all or j == i:
                    yield k_full[(n_k + j) % 4], (n_k + j) // 4
                if watch_all and j != i:
                    q.append(k_empty[(n_k + j) % 4].arrive)
            n_k += tiles
            for t in range(steps):
                yield q_full[n_l % 3], n_l // 3
                if work:
                    if n_s >= 2:
                        yield s_empty[i][n_s % 2], n_s // 2 - 1
                    q.append(product(k_slot, n_l % 3, n_s % 2, n, t))
                    q.append(s_full[i][n_s % 2].arrive)
                    n_s += 1
                q.append(q_empty[n_l % 3].arrive)
                if work and t == steps - 1:
                    q.append(k_empty[k_slot].arrive)
                n_l += 1
                yield None

    def sums(i, half):
        n_s = n_l = n_h = 0
        for n, (tiles, steps) in enumerate(units):
            work = i < tiles
            for t in range(steps):
                if work:
                    yield s_full[i][n_s % 2], n_s // 2
                yield l_full[n_l % 3], n_l // 3
                expect(lses[n_l % 3], (n, t))
                if work:
                    expect(s_at[i][n_s % 2], (n, t))
                    s_empty[i][n_s % 2].arrive()
                    n_s += 1
                yield None
                l_empty[n_l % 3].arrive()
                n_l += 1
            if not work or steps == 0:
                continue
            if half:
                if n_h > 0:
                    yield half_free[i], n_h - 1
                half_at[i] = n
                half_done[i].arrive()
            else:
                yield half_done[i], n_h
                expect(half_at[i], n)
                half_free[i].arrive()
                out[n, i] = True
            n_h += 1

    def landed():
        return [(k_full[n % 4], n // 4) for n in range(max(0, at[0] - 4), at[0])] + \
               [(q_full[n % 3], n // 3) for n in range(max(0, at[1] - 3), at[1])]

    def drained(i):
        m.queues[f"T{i}"].append(drain[i].arrive)
        return [(drain[i], 0)]

    m.add("loads", ending(loads(), landed, ends))
    m.add("rows", ending(rows(), list, ends))
    for i in (0, 1):
        m.queues[f"T{i}"] = []
        m.add(f"products{i}", ending(products(i), lambda i=i: drained(i), ends))
        for half in (0, 1):
            m.add(f"sums{i}.{half}", ending(sums(i, half), list, ends))
    m.run()
    assert gives_up or len(out) == sum(t for t, s in units if s)


def mass_fails(trials, gives_up=False, **kw):
    for trial in range(trials):
        rnd = random.Random(trial)
        units = [(rnd.choice([1, 1, 2]), rnd.choice([0, 1, 1, 1, 2, 3, 5]))
                 for _ in range(rnd.randint(1, 14))]
        who = rnd.choice(["loads", "rows", "products0", "products1", "sums0.0", "sums1.1"])
        try:
            mass(trial, units, gives_up=(who, rnd.randint(1, 20)) if gives_up else None, **kw)
        except (Stall, Wrong) as e:
            return trial, e
    return None


def test_mass_reads_the_keys_of_its_unit():
    assert mass_fails(1500) is None


def test_model_catches_a_mass_warp_that_skips_a_key_tile():
    """A warp that does not wait for the K tiles it does not read falls behind
    the slots' phases: the parity of a use before then passes for its own."""
    assert mass_fails(3000, watch_all=False) is not None


def test_mass_leaves_nothing_behind_when_a_wait_runs_out():
    assert mass_fails(1500, gives_up=True) is None
    assert mass_fails(1500, gives_up=True, ends=False) is not None


# ---------------------------------------------------------------------------
# One wait of a warp whose limit runs out while the phase completes
# ---------------------------------------------------------------------------

def answers(seed, votes):
    """What each of a warp's lanes gets from one wait.  A lane's probe sees the
    phase if it has completed by then; lanes probe, and read the time, at moments
    of their own."""
    rnd = random.Random(seed)
    done_at, limit = rnd.uniform(0, 30), 20.0
    first = [rnd.uniform(0, 1) for _ in range(32)]
    got = [True if t >= done_at else None for t in first]
    t = 1.0
    while any(g is None for g in got):
        left = [n for n in range(32) if got[n] is None]
        for n in left:
            if t + rnd.uniform(0, 1) >= done_at:
                got[n] = True
        t += 1.0
        left = [n for n in left if got[n] is None]
        over = [n for n in left if t + rnd.uniform(0, 1) - first[n] > limit]
        t += 1.0
        if votes and over:       # one last probe, which goes for all that are left
            there = any(t + rnd.uniform(0, 1) >= done_at for _ in left)
            for n in left:
                got[n] = there
        elif not votes:
            for n in over:
                got[n] = False
    return got


def test_a_warp_leaves_a_wait_with_one_answer():
    seen = [set(answers(seed, votes=True)) for seed in range(5000)]
    assert all(len(s) == 1 for s in seen) and {True} in seen and {False} in seen


def test_model_catches_lanes_that_decide_alone():
    assert any(len(set(answers(seed, votes=False))) > 1 for seed in range(5000))
