"""The barriers of k_prompt (csrc/prompt_attn.cuh) as a model on the CPU: its warps take turns in any order, and any wait may
run out.  No wait passes too early; no arrival is more than a barrier expects (which is undefined), not after a lost wait
either; every warp comes to its end, and no copy is in flight there."""
import random

import pytest


class Bar:
    """An mbarrier: pending arrivals and bytes of a phase."""

    def __init__(self, n, name):
        self.n = self.pending = n
        self.phase = self.bytes = 0
        self.name = name

    def over(self, parity):
        return (self.phase & 1) != (parity & 1)

    def arrive(self, k=1):
        assert self.pending >= k, ("more arrivals than are pending", self.name)
        self.pending -= k
        self.settle()

    def settle(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, self.n


class Ring:
    def __init__(self, stages, i=0):
        self.stages, self.i = stages, i

    st = property(lambda self: self.i % self.stages)
    use = property(lambda self: self.i // self.stages)

    def skip(self, n=1):
        self.i += n

    def copy(self):
        return Ring(self.stages, self.i)


class Meet:
    """A named barrier of n warps that says whether any of them is lost."""

    def __init__(self, n):
        self.n, self.here, self.any, self.turn, self.said = n, 0, False, 0, {}

    def come(self, lost):
        turn = self.turn
        self.here += 1
        self.any |= lost
        if self.here == self.n:
            self.said[turn] = self.any
            self.here, self.any, self.turn = 0, False, turn + 1
        while turn not in self.said:
            yield
        return self.said[turn]


def run(MT, C, ST, items, rng, runs_out=0.0, mistake=None):
    full, empty = [Bar(1, "full") for _ in range(ST)], [Bar(MT, "empty") for _ in range(ST)]
    qf, qe, of, oe = ([Bar(n, name) for _ in range(MT)] for n, name in ((1, "qf"), (1, "qe"), (1, "of"), (2, "oe")))
    sf, pf = [Bar(1, "sf") for _ in range(2)], [[Bar(2, "pf") for _ in range(2)] for _ in range(2)]
    pv, near, clean = Bar(1, "pv"), Bar(MT, "near"), Bar(3 - MT, "clean")
    queue = {"copies": [], 0: [], 1: []}       # what ends later, in order: copies, products of either row tile
    holds, gone, flying = [None] * ST, [False], [0]
    meets = [Meet(2) for _ in range(MT)]        # (two of the four warps of a row tile's softmax)
    cleaners = Meet(3 - MT)

    class Role:
        lost = False

        def wait(self, bar, use):
            """For the end of phase number `use`."""
            while not bar.over(use):
                if gone[0] or rng.random() < runs_out:
                    gone[0] = self.lost = True
                    return
                yield
            if not gone[0]:
                assert bar.phase == use + 1, ("a wait that passed too early", bar.name, bar.phase, use)

    def true(x):
        assert gone[0] or x

    def copier():
        me, i, uses = Role(), 0, [0] * MT

        def landed(bar, st=None, what=None):
            def f():
                flying[0] -= 1
                if st is not None:
                    holds[st] = what
                bar.bytes = 0
                bar.settle()
            return f

        def load(bar, *a):
            bar.bytes = 1
            bar.arrive()
            flying[0] += 1
            queue["copies"].append(landed(bar, *a))

        for n, w in enumerate(items):
            if gone[0]:
                break

            def query(t):
                if w["hi"][t] <= w["lo"][t]:
                    return
                if uses[t]:
                    yield from me.wait(qe[t], uses[t] - 1)
                if gone[0]:
                    return
                load(qf[t])
                uses[t] += 1

            def keys(kind, j):
                nonlocal i
                for c in range(C):
                    if i >= ST:
                        yield from me.wait(empty[i % ST], i // ST - 1)
                    if gone[0]:
                        return
                    load(full[i % ST], i % ST, (kind, n, j, c))
                    i += 1
            yield from query(0)
            for j in range(w["j0"], w["j1"]):
                if gone[0]:
                    break
                yield from keys("K", j)
                if MT == 2 and j == w["j0"]:
                    yield from query(1)
                yield from keys("V", j)
            for o in range(w["outs"]):
                if gone[0]:
                    break
                if i >= ST:
                    yield from me.wait(empty[i % ST], i // ST - 1)
                if gone[0] and mistake != "arrives behind a lost wait":
                    break
                holds[i % ST] = ("O", n, o)
                full[i % ST].arrive()
                i += 1
                yield
        if gone[0] and mistake == "leaves its copies":
            return
        for bar, use in [(qf[t], uses[t] - 1) for t in range(MT) if uses[t]] + [(full[x % ST], x // ST) for x in range(max(0, i - ST), i)]:
            while not bar.over(use):
                yield

    def products(t):
        me = Role()
        ks, vs = Ring(ST), Ring(ST, C)
        s = dict(queries=0, outs=0, weights=0, buf=0, unread=False, cleaned=0)

        def commit(bar):
            queue[t].append(bar.arrive)

        def scores(n, w, j):
            mine = w["lo"][t] <= j < w["hi"][t]
            if mine and j == w["lo"][t]:
                yield from me.wait(qf[t], s["queries"])
                s["queries"] += 1
            for c in range(C):
                yield from me.wait(full[ks.st], ks.use)
                true(holds[ks.st] == ("K", n, j, c))
                if mine:
                    queue[t].append(lambda st=ks.st, what=("K", n, j, c): true(holds[st] == what))
                    if c == C - 1:
                        commit(sf[t if MT == 2 else s["buf"]])
                    commit(empty[ks.st])
                else:
                    empty[ks.st].arrive()
                ks.skip()
                yield
            ks.skip(C)
            if mine and j + 1 == w["hi"][t]:
                commit(qe[t])
            if MT == 1:
                s["buf"] ^= 1

        def sums(n, w, j):
            mine, unclean = w["lo"][t] <= j < w["hi"][t], j >= w["up"] or j < w["down"]
            if unclean:
                near.arrive()
            yield
            if mine and j == w["lo"][t] and s["unread"]:
                yield from me.wait(oe[t], s["outs"] - 1)
            if unclean:
                yield from me.wait(clean, s["cleaned"])
                s["cleaned"] += 1
            for c in range(C):
                yield from me.wait(full[vs.st], vs.use)
                true(holds[vs.st] == ("V", n, j, c))
                for half in range(2):
                    if mine and c == 0:
                        yield from me.wait(pf[t if MT == 2 else s["weights"] & 1][half], s["weights"] if MT == 2 else s["weights"] >> 1)
                if mine:
                    queue[t].append(lambda st=vs.st, what=("V", n, j, c): true(holds[st] == what))
                    if c == C - 1 and j + 1 == w["hi"][t]:
                        commit(of[t])
                    commit(empty[vs.st])
                else:
                    empty[vs.st].arrive()
                vs.skip()
                yield
            vs.skip(C)
            if MT == 1:
                commit(pv)
            if mine:
                s["weights"] += 1
                if j + 1 == w["hi"][t]:
                    s["outs"], s["unread"] = s["outs"] + 1, True
        live = [(n, w) for n, w in enumerate(items) if w["j1"] > w["j0"]]
        if live:
            yield from scores(*live[0], live[0][1]["j0"])
        for x, (n, w) in enumerate(live):
            if me.lost:
                break
            j = w["j0"]
            while j + 1 < w["j1"] and not me.lost:
                if MT == 1:
                    yield from scores(n, w, j + 1)
                yield from sums(n, w, j)
                if MT == 2:
                    yield from scores(n, w, j + 1)
                j += 1
            yield from sums(n, w, j)
            ks.skip(w["outs"])
            vs.skip(w["outs"])
            if x + 1 < len(live):
                yield from scores(*live[x + 1], live[x + 1][1]["j0"])
            if s["unread"] and not w["hi"][t]:
                yield from me.wait(oe[t], s["outs"] - 1)
                s["unread"] = False
    marks = {}

    def cleaner():
        me, told, vs, gen = Role(), 0, Ring(ST, C), 0
        for n, w in enumerate(items):
            if w["j1"] <= w["j0"]:
                continue
            for j in range(w["j0"], w["j1"]):
                at = vs.copy()
                vs.skip(2 * C)
                if not (j >= w["up"] or j < w["down"]):
                    continue
                yield from me.wait(near, told)
                told += 1
                marks[gen] = n
                if (yield from cleaners.come(me.lost)):
                    return
                for c in range(C):
                    yield from me.wait(full[at.st], at.use)
                    true(holds[at.st] == ("V", n, j, c))
                    yield
                    true(holds[at.st] == ("V", n, j, c))
                    at.skip()
                clean.arrive()
            vs.skip(w["outs"])
            gen ^= 1

    def softmax(t, first):
        me, tiles, outs, os, gen, owed = Role(), 0, 0, Ring(ST), 1, []

        def release():
            while owed:
                at, n = owed.pop()
                for _ in range(C):
                    true(holds[at.st] is not None and holds[at.st][:2] == ("O", n))
                    if mistake == "several at once":
                        empty[at.st].arrive(MT)
                    else:
                        for _ in range(MT):
                            empty[at.st].arrive()
                    at.skip()
        for n, w in enumerate(items):
            if w["j1"] > w["j0"]:
                gen ^= 1
            ja, jb = w["lo"][t], w["hi"][t]
            if jb <= ja:
                release()
            for j in range(ja, jb):
                buf = t if MT == 2 else tiles & 1
                yield from me.wait(sf[buf], tiles if MT == 2 else tiles >> 1)
                if me.lost:
                    break
                if MT == 1 and j > ja and rng.random() < 0.3:
                    yield from me.wait(pv, tiles - 1)
                for half in range(2):
                    yield
                    pf[buf][half].arrive()
                release()
                tiles += 1
            start = os.i
            os.skip(2 * C * (w["j1"] - w["j0"]))
            if t and w["hi"][0] > w["lo"][0]:
                os.skip(C)
            if jb > ja:
                yield from me.wait(of[t], outs)
                outs += 1
                hidden = any(j >= w["up"] or j < w["down"] for j in range(ja, jb))
                true(not hidden or marks.get(gen) == n)
                o0 = os.copy()
                for _ in range(C):
                    yield from me.wait(full[os.st], os.use)
                    true(holds[os.st] is not None and holds[os.st][:2] == ("O", n))
                    os.skip()
                yield
                true(not hidden or marks.get(gen) == n)
                oe[t].arrive()
                if (yield from meets[t].come(me.lost)):
                    break
                if first:
                    owed.append((o0, n))
                    if rng.random() < 0.4:
                        release()
            os.i = start + 2 * C * (w["j1"] - w["j0"]) + w["outs"]
        release()

    roles = [copier()] + [cleaner() for _ in range(3 - MT)] + [products(t) for t in range(MT)] + \
        [softmax(t, first) for t in range(MT) for first in (True, False)]
    weight, pace = [rng.random() ** 3 + 0.01 for _ in roles], {k: rng.random() ** 3 + 0.01 for k in queue}
    alive = list(range(len(roles)))
    for _ in range(400000):
        if not alive and not any(queue.values()):
            return gone[0]
        busy = [k for k in queue if queue[k]]
        kind, x = rng.choices([("role", a) for a in alive] + [("end", k) for k in busy], [weight[a] for a in alive] + [pace[k] for k in busy])[0]
        if kind == "end":
            queue[x].pop(0)()
            continue
        try:
            next(roles[x])
        except StopIteration:
            alive.remove(x)
            assert alive or not flying[0], "a copy outlives the kernel"
    raise AssertionError(("stuck", alive))


def item(MT, C, rng):
    if rng.random() < 0.1:
        return dict(j0=0, j1=0, lo=[0] * MT, hi=[0] * MT, up=0, down=0, outs=0)
    j0, steps = rng.choice([0, 0, 0, 3]), rng.choice([1, 1, 2, 3, 5, 8])
    lo, hi = [j0] * MT, [j0 + steps] * MT
    if MT == 2:
        r = rng.random()
        if r < 0.3:
            lo[1] = hi[1] = 0
        elif r < 0.4:
            lo[0] = hi[0] = 0
        elif r < 0.7 and steps > 1:
            hi[0] -= 1
        if hi[0] > lo[0] and hi[1] > lo[1] + 1 and lo[1] + 1 <= hi[0] and rng.random() < 0.3:
            lo[1] += 1
    on = [t for t in range(MT) if hi[t] > lo[t]]
    j0, j1 = min(lo[t] for t in on), max(hi[t] for t in on)
    return dict(j0=j0, j1=j1, lo=lo, hi=hi, up=max(j0, j1 - rng.choice([0, 1, 2, 2])), down=min(j1, j0 + rng.choice([0, 0, 1, 2])),
                outs=C * len(on))


SHAPES = [(2, 1, 5), (2, 1, 8), (1, 2, 5)]      # row tiles, stages of a tile of keys, stages of the ring


def case(seed, **kw):
    rng = random.Random(seed)
    MT, C, ST = rng.choice(SHAPES)
    return run(MT, C, ST, [item(MT, C, rng) for _ in range(rng.randint(1, 8))], rng, **kw)


def test_every_order():
    assert not any(case(seed) for seed in range(300))


def test_waits_that_run_out():
    lost = sum(case(seed, runs_out=1e-3) for seed in range(600))
    assert lost > 200


@pytest.mark.parametrize("mistake", ["several at once", "arrives behind a lost wait", "leaves its copies"])
def test_the_model_sees_mistakes(mistake):
    seen = 0
    for seed in range(2000):
        try:
            case(seed, runs_out=1e-3, mistake=mistake)
        except AssertionError as e:
            assert "stuck" not in str(e)
            seen += 1
            if seen == 3:
                return
    raise AssertionError("not seen")
