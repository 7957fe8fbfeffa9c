"""The hand-offs of the shared-prefix decode kernel when a wait expires, as a model.

The roles of pa_prefix_impl.cuh -- copies, conversions, MMA issue, softmax -- run as
generators over the kernel's barriers, in random order, with random waits expiring and a
copy that never lands.  Whatever happens, every role comes to its end (a barrier that
only some of the softmax warps reach would hold a GPU for good), no MMA goes by a tile
record that may not be there, no wait passes a phase
that it does not mean, and a record is not overwritten while a live role needs it."""
import random

import pytest

RING = 16  # tile records


class Fault(Exception):
    pass


class Bar:
    def __init__(self, count, name):
        self.count = self.left = count
        self.phase, self.name, self.pending = 0, name, 0

    def arrive(self):
        if self.left <= 0:
            raise Fault(f"{self.name}: arrived at too often")
        self.left -= 1
        self.turn()

    def turn(self):
        if self.left == 0 and self.pending == 0:
            self.phase += 1
            self.left = self.count


def simulate(seed, agree=True, own_shape=True):
    """agree: the softmax warps leave together; own_shape: after an expired wait MMAs go by no tile's record."""
    rnd = random.Random(seed)
    n, nk, nv = rnd.randint(1, 14), rnd.choice([2, 4, 6, 8, 10]), rnd.choice([2, 4, 6, 8, 10])
    first = [True] + [rnd.random() < 0.35 for _ in range(n)]
    last = [j + 1 == n or first[j + 1] for j in range(n)]
    wide = [rnd.random() < 0.4 for _ in range(n + 1)]  # by piece
    raises = [rnd.random() < 0.25 for _ in range(n)]
    stuck = (rnd.choice("kv"), rnd.randrange(2 * n)) if rnd.random() < 0.8 else None  # a stage that never lands
    early = rnd.choice([0.0, 0.0, 0.002, 0.02])  # chance that a blocked wait expires although others go on

    bars = lambda name, count, m: [Bar(count, f"{name}{i}") for i in range(m)]  # noqa: E731
    raw = {"k": bars("kraw_full", 1, nk), "v": bars("vraw_full", 1, nv)}
    free = {"k": bars("kraw_empty", 4, nk), "v": bars("vraw_empty", 4, nv)}
    ku_full, ku_empty, vu_full, vu_empty = bars("ku_full", 4, 2), bars("ku_empty", 1, 2), bars("vu_full", 4, 2), bars("vu_empty", 1, 2)
    s_full, s_empty, p_full, pv_done = bars("s_full", 1, 2), bars("s_empty", 8, 2), bars("p_full", 8, 2), bars("pv_done", 1, 2)
    q_full, q_empty, o_free = bars("q_full", 8, 2), bars("q_empty", 1, 2), bars("o_free", 8, 2)
    tiles = [None] * RING
    landing, commits_s, commits_p = [], [], []
    aborted = [False]

    def record(j):
        if tiles[j % RING] != j:
            raise Fault(f"record of tile {j} is {tiles[j % RING]}")

    # A wait: yields until its phase is over (True) or it expires (False).
    def wait(bar, parity, phase):
        while True:
            if (bar.phase & 1) != parity:
                if bar.phase != phase + 1:
                    raise Fault(f"{bar.name}: phase {bar.phase} taken for {phase + 1}")
                return True
            if (yield "wait"):
                aborted[0] = True
                return False

    def copy(kind):
        ns = nk if kind == "k" else nv
        for j in range(n):
            if kind == "k":
                tiles[j % RING] = j
            yield None
            for h in range(2):
                s, use = (2 * j + h) % ns, (2 * j + h) // ns
                if use and not (yield from wait(free[kind][s], (use - 1) & 1, use - 1)):
                    return
            for h in range(2):
                s = (2 * j + h) % ns
                raw[kind][s].pending += 1
                raw[kind][s].arrive()
                if stuck != (kind, 2 * j + h):
                    landing.append(raw[kind][s])
                yield None

    def convert_k(kd, quarter):
        piece = 0
        for j in range(n):
            stage = 2 * j + (quarter >> 1)
            s, use = stage % nk, stage // nk
            if j > 0:
                if not (yield from wait(raw["k"][s], use & 1, use)):
                    return
                record(j)
            if first[j]:
                if piece > 1 and not (yield from wait(q_empty[piece & 1], ((piece >> 1) - 1) & 1, (piece >> 1) - 1)):
                    return
                if piece > 0 and (wide[piece] or wide[piece - 1]) and \
                        not (yield from wait(q_empty[(piece - 1) & 1], ((piece - 1) >> 1) & 1, (piece - 1) >> 1)):
                    return
            if j > 0:
                if not (yield from wait(ku_empty[kd], (j - 1) & 1, j - 1)):
                    return
            elif not (yield from wait(raw["k"][s], 0, 0)):
                return
            yield None
            free["k"][s].arrive()
            ku_full[kd].arrive()
            yield None
            if first[j]:
                q_full[piece & 1].arrive()
                piece += 1
                yield None

    def convert_v(vh):
        for j in range(n):
            stage = 2 * j + vh
            s, use = stage % nv, stage // nv
            if not (yield from wait(raw["v"][s], use & 1, use)):
                return
            if j > 0 and not (yield from wait(vu_empty[vh], (j - 1) & 1, j - 1)):
                return
            free["v"][s].arrive()
            yield None
            vu_full[vh].arrive()
            yield None

    def mma(is_s):
        dead, piece = False, 0

        def need(bar, parity, phase):
            nonlocal dead
            if dead:  # a wait after one that expired: its phases mean nothing any more
                yield None
            elif not (yield from wait(bar, parity, phase)):
                dead = True

        def issue(j, bars_to):
            if not (dead and own_shape):
                record(j)
            if not dead:
                bars_to[0].extend(bars_to[1])

        for j in range(n):
            b = j & 1
            if is_s:
                yield from need(ku_full[0], b, j)
                if not dead:
                    record(j)
                if first[j]:
                    yield from need(q_full[piece & 1], (piece >> 1) & 1, piece >> 1)
                    piece += 1
                if j >= 2:
                    yield from need(s_empty[b], ((j >> 1) - 1) & 1, (j >> 1) - 1)
                issue(j, (commits_s, [ku_empty[0]]))
                yield from need(ku_full[1], b, j)
                issue(j, (commits_s, [ku_empty[1], s_full[b]] + ([q_empty[(piece - 1) & 1]] if last[j] else [])))
            else:
                yield from need(p_full[b], (j >> 1) & 1, j >> 1)
                if not dead:
                    record(j)
                if first[j]:
                    if piece > 1:
                        yield from need(o_free[piece & 1], ((piece >> 1) - 1) & 1, (piece >> 1) - 1)
                    if piece > 0 and (wide[piece] or wide[piece - 1]):
                        yield from need(o_free[(piece - 1) & 1], ((piece - 1) >> 1) & 1, (piece - 1) >> 1)
                    piece += 1
                for h in range(2):
                    yield from need(vu_full[h], b, j)
                    issue(j, (commits_p, [vu_empty[h]] + ([pv_done[b]] if h else [])))
            yield None

    # The softmax warps' barrier: every generation is met by all eight, in one form.
    meeting = {"here": [], "generation": 0, "any": False, "results": {}}
    quit_flag = [0, 0]

    def meet(form, x=False):
        g = meeting["generation"]
        meeting["here"].append(form)
        meeting["any"] |= x
        if len(meeting["here"]) == 8:
            if len(set(meeting["here"])) > 1:
                raise Fault("one barrier in two forms")
            meeting["results"][g] = meeting["any"]
            meeting.update(here=[], generation=g + 1, any=False)
        while meeting["generation"] == g:
            yield "meet"
        return meeting["results"][g]

    def softmax(w):
        live = True

        def alive(bar, parity, phase):
            nonlocal live
            if live:
                live = yield from wait(bar, parity, phase)

        def info(j, what):  # what a warp believes of the tile
            if live or tiles[j % RING] == j:
                record(j)
                return what[j]
            if agree:
                raise Fault("a record that may not be there is read")
            return rnd.random() < 0.5

        piece = 0
        for j in range(n + 1):
            if j < n:
                yield from alive(s_full[j & 1], (j >> 1) & 1, j >> 1)
                if not live and agree:
                    quit_flag[j & 1] = 1
                    yield from meet("or", True)
                    return
                is_first = info(j, first)
                for once in range(2):
                    if is_first or once:
                        if j > 0 and (yield from meet("or")):
                            return
                        if (yield from meet("or")):
                            return
                        yield from meet("sync")
                        if not is_first:
                            yield from alive(pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, (j - 1) >> 1)
                    if j > 1 and live:
                        yield from alive(pv_done[j & 1], ((j >> 1) - 1) & 1, (j >> 1) - 1)
                    if is_first or once:
                        break
                    if not live and agree:
                        quit_flag[j & 1] = 1
                    again = yield from meet("or", raises[j] or (agree and not live))
                    if again and quit_flag[j & 1] and agree:
                        return
                    if not again:
                        break
                yield None
                if live:
                    p_full[j & 1].arrive()
                    s_empty[j & 1].arrive()
                yield None
            if j > 0 and info(j - 1, last):
                yield from alive(pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, (j - 1) >> 1)
                yield None
                if live:
                    o_free[piece & 1].arrive()
                piece += 1
            if j < n and info(j, last):
                yield from meet("sync")
                yield from meet("sync")

    roles = {"copy k": copy("k"), "copy v": copy("v"), "s": mma(True), "pv": mma(False)}
    for w in range(8):
        roles[f"k{w}"], roles[f"v{w}"], roles[f"softmax {w}"] = convert_k(w >> 2, w & 3), convert_v(w >> 2), softmax(w)
    state = {}  # what the role yielded last
    quiet = 0  # turns since anything moved
    snapshot = None
    while roles:
        if landing and rnd.random() < 0.5:
            bar = landing.pop(rnd.randrange(len(landing)))
            bar.pending -= 1
            bar.turn()
        for queue in (commits_s, commits_p):
            if queue and rnd.random() < 0.5:
                queue.pop(0).arrive()
        name = rnd.choice(list(roles))
        # expiry: when all stand still, after an abort, or now and then
        expire = state.get(name) == "wait" and (quiet > 400 or (aborted[0] and rnd.random() < 0.05) or rnd.random() < early)
        try:
            state[name] = roles[name].send(expire) if name in state else next(roles[name])
        except StopIteration:
            del roles[name]
            state.pop(name, None)
        now = (tuple(sorted(state.items(), key=str)), len(landing), len(commits_s), len(commits_p), meeting["generation"], len(meeting["here"]),
               sum(b.phase * 16 + b.left for bs in (*raw.values(), *free.values(), ku_full, ku_empty, vu_full, vu_empty, s_full, s_empty, p_full,
                                                    pv_done, q_full, q_empty, o_free) for b in bs))
        quiet = quiet + 1 if now == snapshot else 0
        snapshot = now
        if quiet > 5000:
            raise Fault("held for good: " + ", ".join(f"{k} {v}" for k, v in state.items()))
    return stuck is None and not aborted[0]


def test_every_role_ends():
    clean = sum(simulate(seed) for seed in range(250))
    assert 8 < clean < 190  # some runs without an expired wait, many with


@pytest.mark.parametrize("without", ["agree", "own_shape"])
def test_the_model_sees_what_each_rule_is_for(without):
    faults = 0
    for seed in range(100):
        try:
            simulate(seed, **{without: False})
        except Fault:
            faults += 1
    assert faults > 5
