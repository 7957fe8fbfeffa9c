"""The hand-offs of the prompts' attention kernel when a wait expires, as a model.

The roles of both CTAs of a pair in pa_prompt.cu -- copies of K and of V, word of the second's copies, MMA issue, query rows and results, softmax -- run as
generators over the kernel's barriers, in random order, with random waits expiring and a
copy that never lands.  Whatever happens, every role comes to its end (a barrier that only
some of the softmax warps reach would hold a GPU for good), no wait passes a phase that it does
not mean, every stage is used for what was copied into it, and no sums or query rows are
overwritten while they are needed."""
import random

from test_prefix_handoffs import Bar, Fault

STAGES = 5


def simulate(seed, agree=True):
    rnd = random.Random(seed)
    pieces = [rnd.choice([1, 1, 2, 3, 7]) for _ in range(rnd.randint(1, 6))]  # tiles of each
    tiles = [(i, t, m) for i, m in enumerate(pieces) for t in range(m)]
    v_stages = [rnd.randint(1, 2) for _ in tiles]
    n = len(tiles)
    # the order of the stages: K(0), then K(j + 1) before V(j)
    order = [("k", 0, h) for h in range(2)]
    for j in range(n):
        if j + 1 < n:
            order += [("k", j + 1, h) for h in range(2)]
        order += [("v", j, q) for q in range(v_stages[j])]
    stuck = (rnd.randrange(2), rnd.randrange(len(order))) if rnd.random() < 0.8 else None  # a CTA's stage that never lands
    early = rnd.choice([0.0, 0.0, 0.001, 0.01])
    every = []

    def bars(name, count, m):
        got = [Bar(count, f"{name}{i}") for i in range(m)]
        every.extend(got)
        return got

    # of the two CTAs
    full = [bars("full a", 2, STAGES), bars("full b", 1, STAGES)]
    empty, q_empty, s_full, pv_done, l_full = ([bars(f"{name} {c}", count, m) for c in "ab"] for name, count, m in (
        ("empty", 1, STAGES), ("q_empty", 1, 2), ("s_full", 1, 2), ("pv_done", 1, 2), ("l_full", 8, 2)))
    # of the first
    q_full, p_full, (o_free,), (drain,) = bars("q_full", 8, 2), bars("p_full", 16, 2), bars("o_free", 8, 1), bars("drain", 1, 1)
    stage_of, landing, commits, aborted = [[None] * STAGES, [None] * STAGES], [], [], [False, False]
    sums, queries, o_holds = [{}, {}], {}, [None]

    def wait(bar, phase, c):
        while True:
            if (bar.phase & 1) != (phase & 1):
                if bar.phase != phase + 1:
                    raise Fault(f"{bar.name}: phase {bar.phase} taken for {phase + 1}")
                return True
            if (yield ("wait", c)):
                aborted[c] = True
                return False

    def copy(c, kind):  # a warp's stages: K's or V's
        for i, what in enumerate(order):
            if what[0] != kind:
                continue
            s, use = i % STAGES, i // STAGES
            if use and not (yield from wait(empty[c][s], use - 1, c)):
                return
            stage_of[c][s] = what
            full[c][s].pending += 1
            full[c][s].arrive()
            if (c, i) != stuck:
                landing.append(full[c][s])
            yield None

    def forward():
        for i in range(len(order)):
            if not (yield from wait(full[1][i % STAGES], i // STAGES, 1)):
                return
            full[0][i % STAGES].arrive()
            yield None

    def mma():
        used = scored = 0

        def stage(what):
            nonlocal used
            s = used % STAGES
            if not (yield from wait(full[0][s], used // STAGES, 0)):
                return False
            for c in range(2):
                if stage_of[c][s] != what:
                    raise Fault(f"stage {s} holds {stage_of[c][s]}, not {what}")
            commits.append([empty[0][s], empty[1][s]])
            used += 1
            return True

        def score(j):
            nonlocal scored
            i, t, m = tiles[j]
            if t == 0:
                if not (yield from wait(q_full[scored & 1], scored >> 1, 0)):
                    return False
                scored += 1
            if any(queries.get((c, a, i & 1)) != i for c in range(2) for a in range(4)):
                raise Fault("query rows of another piece")
            for h in range(2):
                if not (yield from stage(("k", j, h))):
                    return False
                yield None
            commits.append([x[j & 1] for x in s_full] + ([x[i & 1] for x in q_empty] if t + 1 == m else []))
            return True

        def run():
            if not (yield from score(0)):
                return
            for j, (i, t, m) in enumerate(tiles):
                if j + 1 < n and not (yield from score(j + 1)):
                    return
                if not (yield from wait(p_full[j & 1], j >> 1, 0)):
                    return
                if t == 0 and i > 0 and not (yield from wait(o_free, i - 1, 0)):
                    return
                for q in range(v_stages[j]):
                    if not (yield from stage(("v", j, q))):
                        return
                    yield None
                commits.append([("o", j)] + [x[j & 1] for x in pv_done])
                yield None

        yield from run()
        commits.append([drain])
        while drain.phase == 0:
            yield ("drain", 0)

    def aux(c, a):
        loads, done = 1, 0

        def load():
            nonlocal loads
            if loads == len(pieces):
                return True
            if loads > 1 and not (yield from wait(q_empty[c][loads & 1], (loads >> 1) - 1, c)):
                return False
            queries[c, a, loads & 1] = loads
            yield None
            q_full[loads & 1].arrive()
            loads += 1
            yield None
            return True

        if not (yield from load()):
            return
        for i, m in enumerate(pieces):
            done += m
            j = done - 1
            if not (yield from wait(l_full[c][i & 1], i >> 1, c)) or not (yield from wait(pv_done[c][j & 1], j >> 1, c)):
                return
            for look in range(2):
                if o_holds[0] != j or any(sums[c].get((i & 1, w)) != i for w in range(8)):
                    raise Fault("results overwritten, or of another piece")
                yield None
            o_free.arrive()
            yield None
            if not (yield from load()):
                return

    meeting = [{"here": [], "generation": 0, "any": False, "results": {}} for _ in range(8)]  # of a CTA's quarter
    leave = [[0, 0] for _ in range(8)]
    raises = [[rnd.random() < 0.3 for _ in range(n)] for _ in range(8)]

    def meet(c, form, x=False):
        m = meeting[c]
        g = m["generation"]
        m["here"].append(form)
        m["any"] |= x
        if len(m["here"]) == 2:
            if len(set(m["here"])) > 1:
                raise Fault("one barrier in two forms")
            m["results"][g] = m["any"]
            m.update(here=[], generation=g + 1, any=False)
        while m["generation"] == g:
            yield ("meet", c >> 2)
        return m["results"][g]

    def softmax(c, w):
        live, g = True, 4 * c + (w & 3)
        for j, (i, t, m) in enumerate(tiles):
            live = live and (yield from wait(s_full[c][j & 1], j >> 1, c))
            if not live:
                if not agree:
                    return
                leave[g][j & 1] = 1
            up = yield from meet(g, "or", t == 0 or raises[g][j])
            if leave[g][j & 1]:
                return
            if up:
                yield from meet(g, "sync")
                if t > 0 and not (yield from wait(pv_done[c][(j - 1) & 1], (j - 1) >> 1, c)):
                    live = False
                    leave[g][(j + 1) & 1] = 1
            yield None
            if live:
                p_full[j & 1].arrive()
            yield None
            if t + 1 == m:
                sums[c][(i & 1, w)] = i
                yield None
                if live:
                    l_full[c][i & 1].arrive()
                yield None

    def first_rows():  # the first piece's, by the softmax warps
        for c in range(2):
            for a in range(4):
                queries[c, a, 0] = 0
                yield None
                q_full[0].arrive()

    roles = {"mma": mma(), "forward": forward(), "first rows": first_rows()}
    for c in range(2):
        for kind in "kv":
            roles[f"copy {c} {kind}"] = copy(c, kind)
        for a in range(4):
            roles[f"aux {c} {a}"] = aux(c, a)
        for w in range(8):
            roles[f"softmax {c} {w}"] = softmax(c, w)
    state, quiet, snapshot = {}, 0, None
    while roles:
        if landing and rnd.random() < 0.5:
            bar = landing.pop(rnd.randrange(len(landing)))
            bar.pending -= 1
            bar.turn()
        if commits and rnd.random() < 0.5:
            for bar in commits.pop(0):
                if isinstance(bar, tuple):
                    o_holds[0] = bar[1]
                else:
                    bar.arrive()
        name = rnd.choice(list(roles))
        held = state.get(name)
        expire = held is not None and held[0] == "wait" and (quiet > 800 or (aborted[held[1]] and rnd.random() < 0.05) or rnd.random() < early)
        try:
            state[name] = roles[name].send(expire) if name in state else next(roles[name])
        except StopIteration:
            del roles[name]
            state.pop(name, None)
        now = (tuple(sorted(state.items(), key=str)), len(landing), len(commits), *((m["generation"], len(m["here"])) for m in meeting),
               sum(b.phase * 16 + b.left for b in every))
        quiet = quiet + 1 if now == snapshot else 0
        snapshot = now
        if quiet > 10000:
            raise Fault("held for good: " + ", ".join(f"{k} {v}" for k, v in state.items()))
    return stuck is None and not any(aborted)


def test_every_role_ends():
    clean = sum(simulate(seed) for seed in range(100))
    assert 4 < clean < 76  # some runs without an expired wait, many with


def test_the_model_sees_what_leaving_together_is_for():
    faults = 0
    for seed in range(100):
        try:
            simulate(seed, agree=False)
        except Fault:
            faults += 1
    assert faults > 5
