"""The hand-offs of the prompts' attention kernel when a wait expires, as a model.

The roles of pa_prompt.cu -- copies, MMA issue, query rows and results, softmax -- run as
generators over the kernel's barriers, in random order, with random waits expiring and a
copy that never lands.  Whatever happens, every role comes to its end (a barrier that only
some of the softmax warps reach would hold a GPU for good), no wait passes a phase that it does
not mean, every stage is used for what was copied into it, and no sums or query rows are
overwritten while they are needed."""
import random

from test_prefix_handoffs import Bar, Fault

STAGES = 9


def simulate(seed, agree=True):
    rnd = random.Random(seed)
    pieces = [rnd.choice([1, 1, 2, 3, 7]) for _ in range(rnd.randint(1, 7))]  # tiles of each
    tiles = [(i, t, m) for i, m in enumerate(pieces) for t in range(m)]
    v_stages = [rnd.randint(1, 4) for _ in tiles]
    n = len(tiles)
    raises = [rnd.random() < 0.3 for _ in range(n)]
    # the order of the stages: of a piece K(0), then K(j + 1) before V(j)
    order, j0 = [], 0
    for m in pieces:
        order += [("k", j0, q) for q in range(4)]
        for t in range(m):
            if t + 1 < m:
                order += [("k", j0 + t + 1, q) for q in range(4)]
            order += [("v", j0 + t, q) for q in range(v_stages[j0 + t])]
        j0 += m
    stuck = rnd.randrange(len(order)) if rnd.random() < 0.8 else None  # a stage that never lands
    early = rnd.choice([0.0, 0.0, 0.002, 0.02])
    bars = lambda name, count, m: [Bar(count, f"{name}{i}") for i in range(m)]  # noqa: E731
    full, empty = bars("full", 1, STAGES), bars("empty", 1, STAGES)
    q_full, q_empty, o_free = Bar(4, "q_full"), Bar(1, "q_empty"), Bar(4, "o_free")
    s_full, p_full, pv_done, l_full = bars("s_full", 1, 2), bars("p_full", 8, 2), bars("pv_done", 1, 2), bars("l_full", 8, 2)
    drain = Bar(1, "drain")
    stage_of, landing, commits, aborted = [None] * STAGES, [], [], [False]
    sums, queries, o_holds = {}, {}, [None]  # parity -> pieces of each warp; of each aux warp; tile that O holds

    def wait(bar, phase):
        while True:
            if (bar.phase & 1) != (phase & 1):
                if bar.phase != phase + 1:
                    raise Fault(f"{bar.name}: phase {bar.phase} taken for {phase + 1}")
                return True
            if (yield "wait"):
                aborted[0] = True
                return False

    def copy():
        for i, what in enumerate(order):
            s, use = i % STAGES, i // STAGES
            if use and not (yield from wait(empty[s], use - 1)):
                return
            stage_of[s] = what
            full[s].pending += 1
            full[s].arrive()
            if i != stuck:
                landing.append(full[s])
            yield None

    def mma():
        used = 0

        def stage(what):
            nonlocal used
            s = used % STAGES
            if not (yield from wait(full[s], used // STAGES)):
                return False
            if stage_of[s] != what:
                raise Fault(f"stage {s} holds {stage_of[s]}, not {what}")
            commits.append([empty[s]])
            used += 1
            return True

        def score(j):
            i, t, m = tiles[j]
            if any(queries.get(a) != i for a in range(4)):
                raise Fault("query rows of another piece")
            for q in range(4):
                if not (yield from stage(("k", j, q))):
                    return False
                yield None
            commits.append([s_full[j & 1]] + ([q_empty] if t + 1 == m else []))
            return True

        def run():
            for j, (i, t, m) in enumerate(tiles):
                if t == 0:
                    if not (yield from wait(q_full, i)) or not (yield from score(j)):
                        return
                if t + 1 < m and not (yield from score(j + 1)):
                    return
                if not (yield from wait(p_full[j & 1], j >> 1)):
                    return
                if t == 0 and i > 0 and not (yield from wait(o_free, i - 1)):
                    return
                for q in range(v_stages[j]):
                    if not (yield from stage(("v", j, q))):
                        return
                    yield None
                commits.append([("o", j), pv_done[j & 1]])
                yield None

        yield from run()
        commits.append([drain])
        while drain.phase == 0:
            yield "drain"

    def aux(a):
        done = 0
        for i in range(len(pieces) + 1):
            if i < len(pieces):
                if i and not (yield from wait(q_empty, i - 1)):
                    return
                queries[a] = i
                yield None
                q_full.arrive()
                yield None
            if i:
                b, j = i - 1, done - 1
                if not (yield from wait(l_full[b & 1], b >> 1)) or not (yield from wait(pv_done[j & 1], j >> 1)):
                    return
                if o_holds[0] != j or any(sums.get((b & 1, w)) != b for w in range(8)):
                    raise Fault("results of another piece")
                yield None
                if o_holds[0] != j or any(sums.get((b & 1, w)) != b for w in range(8)):
                    raise Fault("results overwritten while they are read")
                o_free.arrive()
                yield None
            if i < len(pieces):
                done += pieces[i]

    meeting = {"here": [], "generation": 0, "any": False, "results": {}}
    leave = [0, 0]

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
        for j, (i, t, m) in enumerate(tiles):
            live = live and (yield from wait(s_full[j & 1], j >> 1))
            if not live:
                if not agree:
                    return
                leave[j & 1] = 1
            up = yield from meet("or", t == 0 or raises[j])
            if leave[j & 1]:
                return
            if up:
                yield from meet("sync")
                if t > 0 and not (yield from wait(pv_done[(j - 1) & 1], (j - 1) >> 1)):
                    live = False
                    leave[(j + 1) & 1] = 1
            yield None
            if live:
                p_full[j & 1].arrive()
            yield None
            if t + 1 == m:
                sums[(i & 1, w)] = i
                yield None
                if live:
                    l_full[i & 1].arrive()
                yield None

    roles = {"copy": copy(), "mma": mma()}
    for a in range(4):
        roles[f"aux {a}"] = aux(a)
    for w in range(8):
        roles[f"softmax {w}"] = softmax(w)
    state, quiet, snapshot = {}, 0, None
    every = [*full, *empty, q_full, q_empty, o_free, *s_full, *p_full, *pv_done, *l_full, drain]
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
        expire = state.get(name) == "wait" and (quiet > 400 or (aborted[0] and rnd.random() < 0.05) or rnd.random() < early)
        try:
            state[name] = roles[name].send(expire) if name in state else next(roles[name])
        except StopIteration:
            del roles[name]
            state.pop(name, None)
        now = (tuple(sorted(state.items(), key=str)), len(landing), len(commits), meeting["generation"], len(meeting["here"]),
               sum(b.phase * 16 + b.left for b in every))
        quiet = quiet + 1 if now == snapshot else 0
        snapshot = now
        if quiet > 5000:
            raise Fault("held for good: " + ", ".join(f"{k} {v}" for k, v in state.items()))
    return stuck is None and not aborted[0]


def test_every_role_ends():
    clean = sum(simulate(seed) for seed in range(250))
    assert 8 < clean < 190  # some runs without an expired wait, many with


def test_the_model_sees_what_leaving_together_is_for():
    faults = 0
    for seed in range(100):
        try:
            simulate(seed, agree=False)
        except Fault:
            faults += 1
    assert faults > 5
