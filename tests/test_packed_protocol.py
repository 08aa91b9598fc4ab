"""Discrete-event models of the barrier protocols of the packed-prompt kernels, checked on CPU.

The blocks of forward_kernel (csrc/packed.cu), dq_kernel and dkv_kernel (csrc/packed_grad.cu) stay for
many work items, and their warps meet only through mbarriers: a scheduling warp that hands out the
items and clears what a tile holds past its sequence's end, a copying thread, two issuing warps, and
the element-wise warps, whose output of one item is written beside the first tile of the next.  A
mistake there hangs or faults on the GPU, where it cannot be tried safely.  The models follow the
kernels' structure (one agent a role, the same barriers and phases; the threads of a role that
arrive together count as one) and run it on random items under random latencies.  For every run they
check that every agent finishes, that no barrier gets more arrivals than its phase counts and no parity
wait is ambiguous, and that nothing is read before it is there or overwritten while it is needed.  The
order in which the two issuers take turns is left out: it is a hint, and the models allow every order.
Planted mistakes have to be reported.
"""
import random

import pytest

from tests._protomodel import Bar, Hazard, Sim, TensorPipe

ITEMS = 4  # places for work items on their way to the other warps (dq_kernel: one)


def check(cond, what):
    if not cond:
        raise Hazard(what)


class Block:
    """What the three kernels share: the items, the ring, the latencies."""

    def __init__(self, seed, items, slots, readers, mutate, places=ITEMS):
        self.rng = random.Random(seed)
        self.sim = Sim(self.rng)
        self.items, self.slots, self.mutate, self.places = items, slots, mutate, places
        self.bar_item = [Bar(f"item{i}", 1) for i in range(places)]
        self.bar_read = [Bar(f"item_read{i}", readers) for i in range(places)]
        self.place = [None] * places
        self.pace = {}

    def product(self, who):
        """How long a product of `who` takes; some are slow all along."""
        pace = self.pace.setdefault(id(who), self.rng.choice([1, 1, 1, 6]))
        return self.rng.uniform(0.2, 0.6) * pace

    def lat(self, lo, hi):
        return ("delay", self.rng.uniform(lo, hi))

    def wait(self, bar, phase):
        return ("wait", lambda: bar.passed(phase))

    def next_item(self, k):
        """A role's wait for item k; yields, then returns the item (None: no more)."""
        yield self.wait(self.bar_item[k % self.places], k // self.places)
        got = self.place[k % self.places]
        check(got[0] == k, "an item was overwritten")
        yield self.lat(0, 0.1)
        self.bar_read[k % self.places].arrive()
        return got[1]

    def publish(self, k):
        if k >= self.places:
            yield self.wait(self.bar_read[k % self.places], k // self.places - 1)
        self.place[k % self.places] = (k, self.items[k] if k < len(self.items) else None)
        self.bar_item[k % self.places].arrive()


class Ring:
    """Places that copies write and products read: each holds (entry, ready, readers left)."""

    def __init__(self, block, name, slots):
        self.b, self.name, self.n = block, name, slots
        self.held = [None] * slots

    def load(self, entry, bar, ready=True, readers=2):
        s = entry % self.n
        check(self.held[s] is None or self.held[s][2] == 0, f"{self.name}: copy over a tile still in use")
        self.held[s] = [entry, False, readers]

        def land():
            self.held[s][1] = ready
            bar.complete_tx(1)
        self.b.sim.at(self.b.rng.uniform(0.2, 3.0), land)

    def cleared(self, entry):
        self.held[entry % self.n][1] = True

    def start(self, entry):
        h = self.held[entry % self.n]
        check(h is not None and h[0] == entry and h[1], f"{self.name}: tile {entry} read before it was there")

    def end(self, entry):
        self.held[entry % self.n][2] -= 1


# ------------------------------------------------------------------------------------ forward
def forward(items, slots, seed, apart, mutate=None):
    """items: (KV tiles of query tile A, of B, whether the last V tile has rows to clear)."""
    b = Block(seed, items, slots, 5, mutate)
    sim, lat, wait = b.sim, b.lat, b.wait
    full = [Bar(f"full{s}", 1) for s in range(slots)]
    empty = [Bar(f"empty{s}", 2) for s in range(slots)]
    tail = [Bar(f"tail{s}", 1) for s in range(slots)]
    if mutate == "one_tail":
        tail = [tail[0]] * slots
    two = lambda name: [Bar(f"{name}{x}", 1) for x in range(2)]  # noqa: E731
    bq, bq_free, bs, bp, bpv, bo = (two(n) for n in ("q", "q_free", "s", "p", "pv", "o_free"))
    ring = Ring(b, "ring", slots)
    q = [None, None]                       # item whose Q is in place, landed
    s_region, p_region = [None, None], [None, None]  # step whose scores (weights) are complete
    pv_ended = [-1, -1]
    o = [None, None]                       # item whose output is in O
    o_read = [True, True]

    def scheduler():
        entries, clear, phase, one, k = 0, None, [0] * slots, 0, 0
        more = True
        while more or clear is not None:
            item = None
            if more:
                yield from b.publish(k)
                item = items[k] if k < len(items) else None
                more = item is not None
            if clear is not None:
                s = clear % slots
                if mutate != "no_clear_wait":
                    yield wait(tail[s], one if mutate == "one_tail" else phase[s])
                one += 1
                phase[s] += 1
                yield lat(0.1, 0.4)
                check(ring.held[s] is not None and ring.held[s][0] == clear, "cleared another tile")
                ring.cleared(clear)
                full[s].arrive()
                clear = None
            if item is not None:
                n = max(item[0], item[1])
                entries += 2 * n
                if n > 0 and item[2]:
                    clear = entries - 1
            k += 1
            yield lat(0, 0.3)

    def copies():
        entry, uses, k = 0, [0, 0], 0
        while (item := (yield from b.next_item(k))) is not None:
            n = max(item[0], item[1])
            for x in range(2):
                if item[x] == 0:
                    continue
                if uses[x] > 0 and mutate != "q_early":
                    yield wait(bq_free[x], uses[x] - 1)
                check(q[x] is None or q[x][2], "Q overwritten while it is read")
                q[x] = [k, False, False]
                uses[x] += 1
                bq[x].arrive(expect=1)

                def land(x=x):
                    q[x][1] = True
                    bq[x].complete_tx(1)
                sim.at(b.rng.uniform(0.2, 2.0), land)
            for i in range(2 * n):
                s = entry % slots
                if entry >= slots:
                    yield wait(empty[s], entry // slots - 1)
                last = item[2] and i == 2 * n - 1
                bar = tail[s] if last else full[s]
                bar.arrive(expect=1)
                ring.load(entry, bar, ready=not last)
                entry += 1
                yield lat(0, 0.1)
            k += 1

    def issuer(x):
        pipe = TensorPipe(sim)
        e, uses, steps, k = 0, 0, 0, 0

        def scores(entry, step, item_no, last):
            def start():
                ring.start(entry)
                check(q[x] is not None and q[x][0] == item_no and q[x][1], "S before its Q")
                if not apart:
                    check(step == 0 or pv_ended[x] >= step - 1, "S over weights that are still read")
                s_region[x] = None
                if not apart:
                    p_region[x] = None

            def end():
                ring.end(entry)
                s_region[x] = step
                if last:
                    q[x][2] = True
            pipe.mma(b.product(pipe), start, end)

        def values(entry, step, item_no, first):
            def start():
                ring.start(entry)
                check(p_region[x] == step, "P V before its weights")
                if first:
                    check(o_read[x], "O overwritten before it was read")
                    o[x], o_read[x] = item_no, False
                check(o[x] == item_no, "P V into another item's O")

            def end():
                ring.end(entry)
                pv_ended[x] = step
            pipe.mma(b.product(pipe), start, end)

        while (item := (yield from b.next_item(k))) is not None:
            nx, n = item[x], max(item[0], item[1])
            if nx > 0:
                yield wait(bq[x], uses)
                yield wait(full[e % slots], e // slots)
                scores(e, steps, k, nx == 1)
                pipe.commit(bs[x])
                pipe.commit(empty[e % slots])
                if nx == 1:
                    pipe.commit(bq_free[x])
            for j in range(nx):
                v = e + 2 * j + 1
                yield wait(full[v % slots], v // slots)
                if j + 1 < nx:
                    yield wait(full[(v + 1) % slots], (v + 1) // slots)
                if j == 0 and uses > 0 and mutate != "no_o_free":
                    yield wait(bo[x], uses - 1)
                yield wait(bp[x], steps + j)
                values(v, steps + j, k, j == 0)
                if j + 1 < nx:
                    scores(v + 1, steps + j + 1, k, j + 2 == nx)
                pipe.commit(bpv[x])
                pipe.commit(empty[v % slots])
                if j + 1 < nx:
                    pipe.commit(bs[x])
                    pipe.commit(empty[(v + 1) % slots])
                    if j + 2 == nx:
                        pipe.commit(bq_free[x])
            for i in range(e + 2 * nx, e + 2 * n):
                if mutate != "no_release":
                    yield wait(full[i % slots], i // slots)
                    ring.end(i)
                    empty[i % slots].arrive()
            e += 2 * n
            steps += nx
            uses += nx > 0
            k += 1

    def softmax(x):
        steps, pending, k, more = 0, None, 0, True
        while more:
            item = yield from b.next_item(k)
            more = item is not None
            nx = item[x] if more else 0
            yield lat(0, 3.0)
            for j in range(-1, nx):
                if j >= 0:
                    yield wait(bs[x], steps)
                    check(s_region[x] == steps, "scores read before they are there")
                    yield lat(0.3, 1.0)
                    if j > 0 and b.rng.random() < 0.3:  # a maximum that grew
                        yield wait(bpv[x], steps - 1)
                        check(pv_ended[x] >= steps - 1, "O rescaled under a running product")
                    check(s_region[x] == steps, "scores overwritten while they are read")
                    check(steps == 0 or pv_ended[x] >= steps - 1, "weights overwritten while they are read")
                    p_region[x] = steps
                    if not apart:
                        s_region[x] = None
                    bp[x].arrive()
                    steps += 1
                if pending is not None and (j == 0 or nx == 0 or bs[x].done <= steps):
                    item_no, last = pending
                    pending = None
                    yield wait(bpv[x], last)
                    check(o[x] == item_no and pv_ended[x] == last, "another item's output written")
                    yield lat(0.2, 1.0)
                    check(o[x] == item_no, "output overwritten while it is read")
                    o_read[x] = True
                    bo[x].arrive()
            if nx > 0:
                pending = (k, steps - 1)
            k += 1

    sim.start("scheduler", scheduler())
    sim.start("copies", copies())
    for x in range(2):
        sim.start(f"issuer{x}", issuer(x))
        sim.start(f"softmax{x}", softmax(x))
    sim.run()


def _pairs(rng):
    out = []
    for _ in range(rng.randrange(1, 14)):
        a, c = rng.choice([(0, 0), (1, 1), (1, 2), (2, 2), (3, 4), (6, 6), (2, 0), (0, 1), (1, 0), (0, 3)])
        out.append((a, c, rng.random() < 0.7))
    return out


@pytest.mark.parametrize("slots,apart", [(4, False), (8, True)])
def test_forward_protocol(slots, apart):
    for seed in range(250):
        forward(_pairs(random.Random(seed)), slots, seed, apart)


@pytest.mark.parametrize("mutate", ["one_tail", "no_clear_wait", "q_early", "no_release", "no_o_free"])
def test_forward_reports(mutate):
    found = 0
    for seed in range(150):
        try:
            forward(_pairs(random.Random(seed)), 4, seed, False, mutate)
        except Hazard:
            found += 1
    assert found > 0


# ------------------------------------------------------------------------------------ dq
def queries(items, keep, passing, seed, mutate=None):
    """dq_kernel.  items: (key tiles, whether the last K tile has rows to clear)."""
    b = Block(seed, items, keep, 4, mutate, places=1)
    sim, lat, wait = b.sim, b.lat, b.wait
    k_full, k_empty = ([Bar(f"{n}{i}", 1) for i in range(keep)] for n in ("k_full", "k_empty"))
    tail = Bar("tail", 1)
    v_full, v_empty = ([Bar(f"{n}{i}", 1) for i in range(passing)] for n in ("v_full", "v_empty"))
    bq, bq_free, bs, bs_read, bdp, bdp_read, bo = (Bar(n, 1) for n in ("q", "q_free", "s", "s_read", "dp", "dp_read", "o_free"))
    bds, bdq = ([Bar(f"{n}{i}", 1) for i in range(2)] for n in ("ds", "dq"))
    ks, vs = Ring(b, "K", keep), Ring(b, "V", passing)
    st = dict(q=None, s=None, dp=None, ds=[None, None], dq_ended=-1, o=None, o_read=True)

    def scheduler():
        tiles, clear, tails, k, more = 0, None, 0, 0, True
        while more or clear is not None:
            item = None
            if more:
                yield from b.publish(k)
                item = items[k] if k < len(items) else None
                more = item is not None
            if clear is not None:
                s = clear % keep
                yield wait(tail, tails)
                tails += 1
                yield lat(0.1, 0.4)
                ks.cleared(clear)
                k_full[s].arrive()
                clear = None
            if item is not None:
                tiles += item[0]
                if item[0] > 0 and item[1]:
                    clear = tiles - 1
            k += 1
            yield lat(0, 0.3)

    def copies():
        tile, uses, k = 0, 0, 0
        while (item := (yield from b.next_item(k))) is not None:
            n = item[0]
            if n > 0:
                if uses > 0:
                    yield wait(bq_free, uses - 1)
                check(st["q"] is None or st["q"][2], "Q overwritten while it is read")
                st["q"] = [k, False, False]
                uses += 1
                bq.arrive(expect=1)

                def land():
                    st["q"][1] = True
                    bq.complete_tx(1)
                sim.at(b.rng.uniform(0.2, 2.0), land)
            for j in range(n):
                kp, vp = tile % keep, tile % passing
                if tile >= keep:
                    yield wait(k_empty[kp], tile // keep - 1)
                last = item[1] and j == n - 1
                bar = tail if last else k_full[kp]
                bar.arrive(expect=1)
                ks.load(tile, bar, ready=not last)
                if tile >= passing:
                    yield wait(v_empty[vp], tile // passing - 1)
                v_full[vp].arrive(expect=1)
                vs.load(tile, v_full[vp], readers=1)
                tile += 1
                yield lat(0, 0.1)
            k += 1

    def first_issuer():
        pipe = TensorPipe(sim)
        step, uses, k = 0, 0, 0

        def product(ring, tile, region, item_no, last=False):
            def start():
                ring.start(tile)
                check(st["q"][0] == item_no and st["q"][1], "a product before its Q")
                check(st[region] is None, f"{region} overwritten before it was read")

            def end():
                ring.end(tile)
                st[region] = tile
                if last:
                    st["q"][2] = True
            pipe.mma(b.product(pipe), start, end)

        while (item := (yield from b.next_item(k))) is not None:
            if item[0] > 0:
                yield wait(bq, uses)
                uses += 1
            for j in range(item[0]):
                yield wait(k_full[step % keep], step // keep)
                if step >= 1 and mutate != "s_unread":
                    yield wait(bs_read, step - 1)
                product(ks, step, "s", k)
                pipe.commit(bs)
                yield wait(v_full[step % passing], step // passing)
                if step >= 1:
                    yield wait(bdp_read, step - 1)
                product(vs, step, "dp", k, j == item[0] - 1)
                pipe.commit(bdp)
                pipe.commit(v_empty[step % passing])
                if j == item[0] - 1:
                    pipe.commit(bq_free)
                step += 1
            k += 1

    def second_issuer():
        pipe = TensorPipe(sim)
        step, uses, k = 0, 0, 0
        while (item := (yield from b.next_item(k))) is not None:
            if item[0] > 0:
                if uses > 0 and mutate != "no_o_free":
                    yield wait(bo, uses - 1)
                uses += 1
            for j in range(item[0]):
                yield wait(k_full[step % keep], step // keep)
                yield wait(bds[step & 1], step // 2)

                def start(step=step, j=j, k=k):
                    ks.start(step)
                    check(st["ds"][step & 1] == step, "dS K before its dS")
                    if j == 0:
                        check(st["o_read"], "dQ overwritten before it was read")
                        st["o"], st["o_read"] = k, False

                def end(step=step):
                    ks.end(step)
                    st["dq_ended"] = step
                pipe.mma(b.product(pipe), start, end)
                pipe.commit(bdq[step & 1])
                pipe.commit(k_empty[step % keep])
                step += 1
            k += 1

    def weights():
        step, pending, k, more = 0, None, 0, True
        while more:
            item = yield from b.next_item(k)
            more = item is not None
            n = item[0] if more else 0
            yield lat(0, 3.0)
            for j in range(-1, n):
                if j >= 0:
                    if step >= 2 and mutate != "ds_unread":
                        yield wait(bdq[step & 1], step // 2 - 1)
                    yield wait(bs, step)
                    check(st["s"] == step, "scores read before they are there")
                    yield lat(0.1, 0.3)
                    st["s"] = None
                    bs_read.arrive()
                    yield lat(0.2, 0.8)
                    yield wait(bdp, step)
                    check(st["dp"] == step, "dP read before it is there")
                    yield lat(0.1, 0.3)
                    st["dp"] = None
                    bdp_read.arrive()
                    yield lat(0.1, 0.4)
                    check(step < 2 or st["dq_ended"] >= step - 2, "dS overwritten while it is read")
                    st["ds"][step & 1] = step
                    bds[step & 1].arrive()
                    step += 1
                if pending is not None and (j == 0 or n == 0 or bs.done <= step):
                    item_no, last = pending
                    pending = None
                    yield wait(bdq[last & 1], last // 2)
                    check(st["o"] == item_no and st["dq_ended"] == last, "another item's dQ written")
                    yield lat(0.1, 0.4)
                    check(st["o"] == item_no, "dQ overwritten while it is read")
                    st["o_read"] = True
                    bo.arrive()
            if n > 0:
                pending = (k, step - 1)
            k += 1

    for name, gen in (("scheduler", scheduler()), ("copies", copies()), ("first", first_issuer()),
                      ("second", second_issuer()), ("weights", weights())):
        sim.start(name, gen)
    sim.run()


def _single(rng):
    return [(rng.choice([0, 1, 1, 1, 2, 3, 5, 9]), rng.random() < 0.7) for _ in range(rng.randrange(1, 16))]


@pytest.mark.parametrize("keep,passing", [(3, 2), (4, 4)])
def test_dq_protocol(keep, passing):
    for seed in range(250):
        queries(_single(random.Random(seed)), keep, passing, seed)


@pytest.mark.parametrize("mutate", ["s_unread", "ds_unread", "no_o_free"])
def test_dq_reports(mutate):
    found = 0
    for seed in range(200):
        try:
            queries(_single(random.Random(seed)), 3, 2, seed, mutate)
        except Hazard:
            found += 1
    assert found > 0


# ------------------------------------------------------------------------------------ dk and dv
def keys(items, slots, seed, apart, mutate=None):
    """dkv_kernel.  items: (query tiles, whether the last one has rows to clear)."""
    b = Block(seed, items, slots, 4, mutate)
    sim, lat, wait = b.sim, b.lat, b.wait
    full = [Bar(f"full{s}", 1) for s in range(slots)]
    empty = [Bar(f"empty{s}", 2) for s in range(slots)]
    tail = Bar("tail", 1)
    kv, kv_free = Bar("kv", 1), Bar("kv_free", 2)
    two = lambda name: [Bar(f"{name}{x}", 1) for x in range(2)]  # noqa: E731
    rows, rows_read, first, packed, second = (two(n) for n in ("rows", "rows_read", "first", "packed", "second"))
    ring = Ring(b, "ring", slots)
    st = dict(kv=None, rows=[None, None], region=[None, None], weights=[None, None], ended=[-1, -1],
              out=[None, None], out_read=[True, True])

    def scheduler():
        step, tails, k = 0, 0, 0
        yield from b.publish(0)
        while k < len(items):
            yield from b.publish(k + 1)
            n, clear = items[k]
            for i in range(n):
                yield lat(0.1, 0.5)
                if step >= 2 and mutate != "rows_unread":
                    yield wait(rows_read[step & 1], step // 2 - 1)
                check(st["rows"][step & 1] is None, "row data overwritten before it was read")
                st["rows"][step & 1] = step
                rows[step & 1].arrive()
                if clear and i == n - 1:
                    yield wait(tail, tails)
                    tails += 1
                    yield lat(0.1, 0.4)
                    for x in range(2):
                        ring.cleared(2 * step + x)
                        full[(2 * step + x) % slots].arrive()
                step += 1
            k += 1

    def copies():
        entry, uses, k = 0, 0, 0
        while (item := (yield from b.next_item(k))) is not None:
            n, clear = item
            if n > 0:
                if uses > 0 and mutate != "kv_early":
                    yield wait(kv_free, uses - 1)
                check(st["kv"] is None or st["kv"][2] == 0, "K and V overwritten while they are read")
                st["kv"] = [k, False, 2]
                uses += 1
                kv.arrive(expect=1)

                def land():
                    st["kv"][1] = True
                    kv.complete_tx(1)
                sim.at(b.rng.uniform(0.2, 2.0), land)
            for i in range(2 * n):
                s = entry % slots
                if entry >= slots:
                    yield wait(empty[s], entry // slots - 1)
                last = clear and i >= 2 * n - 2
                bar = full[s]
                if not last:
                    bar.arrive(expect=1)
                else:
                    bar = tail
                    if not i & 1:
                        bar.arrive(expect=2)
                ring.load(entry, bar, ready=not last)
                entry += 1
                yield lat(0, 0.1)
            k += 1

    def issuer(x):
        pipe = TensorPipe(sim)
        step, uses, k = 0, 0, 0

        def one(entry, at, item_no, last):
            def start():
                ring.start(entry)
                check(st["kv"][0] == item_no and st["kv"][1], "a product before its K or V")
                if not apart:
                    check(at == 0 or st["ended"][x] >= at - 1, "scores over weights that are still read")
                    st["weights"][x] = None
                st["region"][x] = None

            def end():
                ring.end(entry)
                st["region"][x] = at
                if last:
                    st["kv"][2] -= 1
            pipe.mma(b.product(pipe), start, end)

        def two_(entry, at, item_no, begin):
            def start():
                ring.start(entry)
                check(st["weights"][x] == at, "a second product before its weights")
                if begin:
                    check(st["out_read"][x], "dk or dv overwritten before it was read")
                    st["out"][x], st["out_read"][x] = item_no, False

            def end():
                ring.end(entry)
                st["ended"][x] = at
            pipe.mma(b.product(pipe), start, end)

        while (item := (yield from b.next_item(k))) is not None:
            n = item[0]
            if n > 0:
                mine = 2 * step + x
                yield wait(kv, uses)
                yield wait(full[mine % slots], mine // slots)
                one(mine, step, k, n == 1)
                pipe.commit(first[x])
                pipe.commit(empty[mine % slots])
                if n == 1:
                    pipe.commit(kv_free)
            for i in range(n):
                mine, other = 2 * step + 2 + x, 2 * step + 1 - x
                yield wait(full[other % slots], other // slots)
                if i + 1 < n:
                    yield wait(full[mine % slots], mine // slots)
                yield wait(packed[x], step)
                two_(other, step, k, i == 0)
                if i + 1 < n:
                    one(mine, step + 1, k, i + 2 == n)
                pipe.commit(second[x])
                pipe.commit(empty[other % slots])
                if i + 1 < n:
                    pipe.commit(first[x])
                    pipe.commit(empty[mine % slots])
                    if i + 2 == n:
                        pipe.commit(kv_free)
                step += 1
            uses += n > 0
            k += 1

    def weights():
        step, k = 0, 0
        while (item := (yield from b.next_item(k))) is not None:
            n = item[0]
            for _ in range(n):
                yield wait(rows[step & 1], step // 2)
                check(st["rows"][step & 1] == step, "row data read before it is there")
                for x in range(2):
                    yield wait(first[x], step)
                    check(st["region"][x] == step, "scores read before they are there")
                    yield lat(0.2, 0.8)
                    check(st["region"][x] == step, "scores overwritten while they are read")
                    if x == 1:
                        st["rows"][step & 1] = None
                        rows_read[step & 1].arrive()
                    check(step == 0 or st["ended"][x] >= step - 1, "weights overwritten while they are read")
                    st["weights"][x] = step
                    if not apart:
                        st["region"][x] = None
                    packed[x].arrive()
                step += 1
            if n > 0:
                yield lat(0, 3.0)
                for x in range(2):  # (two groups of warps, side by side)
                    yield wait(second[x], step - 1)
                    check(st["out"][x] == k and st["ended"][x] == step - 1, "another item's dk or dv written")
                    yield lat(0.1, 0.6)
                    check(st["out"][x] == k, "dk or dv overwritten while it is read")
                    st["out_read"][x] = True
            k += 1

    for name, gen in (("scheduler", scheduler()), ("copies", copies()), ("issuer0", issuer(0)),
                      ("issuer1", issuer(1)), ("weights", weights())):
        sim.start(name, gen)
    sim.run()


@pytest.mark.parametrize("slots,apart", [(5, False), (8, True)])
def test_dkv_protocol(slots, apart):
    for seed in range(250):
        keys(_single(random.Random(seed)), slots, seed, apart)


@pytest.mark.parametrize("mutate", ["rows_unread", "kv_early"])
def test_dkv_reports(mutate):
    found = 0
    for seed in range(250):
        try:
            keys(_single(random.Random(seed)), 5, seed, False, mutate)
        except Hazard:
            found += 1
    assert found > 0
