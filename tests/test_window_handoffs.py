"""The meetings of the softmax warps at a piece's end in the windowed build of pa_prefix_impl.cuh, as a model.

There the warps meet a third time, and a finished segment's reciprocal sums lie in one array, which is written
after the second meeting of a piece's last tile and read when the next tile's weights are done.  The eight
warps and an MMA issuer run as generators in random order, with waits that expire and an issuer that
stops: every warp comes to its end, every generation of their barrier is met by all in one form, and no
warp writes a result with another piece's sums, or with sums that are not there yet."""
import random

import pytest

from test_prefix_handoffs import Bar, Fault

WARPS, WRITERS = 8, 2  # 64 rows: the first two warps' threads have one each


def simulate(seed, third=True, second=True, agree=True):
    """third, second: the meetings of these numbers take place; agree: the warps leave together."""
    rnd = random.Random(seed)
    n = rnd.randint(1, 14)
    last = [rnd.random() < 0.4 or j + 1 == n for j in range(n)]
    first = [j == 0 or last[j - 1] for j in range(n)]
    raises = [rnd.random() < 0.25 for _ in range(n)]
    whole = [rnd.random() < 0.7 for _ in range(n)]  # of the piece that ends here: the segment's only one
    stop = rnd.randrange(2 * n + 1) if rnd.random() < 0.6 else 2 * n  # products that the issuer completes
    early = rnd.choice([0.0, 0.0, 0.002, 0.02])
    bars = lambda name, count: [Bar(count, f"{name}{i}") for i in range(2)]  # noqa: E731
    s_full, s_empty, p_full, pv_done = bars("s_full", 1), bars("s_empty", 8), bars("p_full", 8), bars("pv_done", 1)
    inv, aborted = [None] * WRITERS, [False]
    meeting = {"here": [], "generation": 0, "any": False, "results": {}}
    quit_flag = [0, 0]

    def wait(bar, phase):
        while True:
            if (bar.phase & 1) != (phase & 1):
                if bar.phase != phase + 1:
                    raise Fault(f"{bar.name}: phase {bar.phase} taken for {phase + 1}")
                return True
            if (yield "wait"):
                aborted[0] = True
                return False

    def issue():
        done = 0
        for j in range(n + 1):
            if j < n:  # S(j)
                if j >= 2 and not (yield from wait(s_empty[j & 1], (j >> 1) - 1)):
                    return
                if done == stop:
                    return
                done += 1
                s_full[j & 1].arrive()
                yield None
            if j > 0:  # PV(j - 1)
                i = j - 1
                if not (yield from wait(p_full[i & 1], i >> 1)):
                    return
                if done == stop:
                    return
                done += 1
                pv_done[i & 1].arrive()
                yield None

    def meet(form, x=False):
        g = meeting["generation"]
        meeting["here"].append(form)
        meeting["any"] |= x
        if len(meeting["here"]) == WARPS:
            if len(set(meeting["here"])) > 1:
                raise Fault("one barrier in two forms")
            meeting["results"][g] = meeting["any"]
            meeting.update(here=[], generation=g + 1, any=False)
        while meeting["generation"] == g:
            yield "meet"
        return meeting["results"][g]

    def softmax(w):
        live = True

        def alive(bar, phase):
            nonlocal live
            if live:
                live = yield from wait(bar, phase)

        for j in range(n + 1):
            if j < n:
                yield from alive(s_full[j & 1], j >> 1)
                if not live:
                    quit_flag[j & 1] = 1
                    if agree:
                        yield from meet("or", True)
                    return
                for once in range(2):
                    if first[j] or once:
                        if j > 0 and (yield from meet("or")):
                            return
                        if (yield from meet("or")):
                            return
                        yield from meet("sync")
                        if not first[j]:
                            yield from alive(pv_done[(j - 1) & 1], (j - 1) >> 1)
                    if j > 1 and live:
                        yield from alive(pv_done[j & 1], (j >> 1) - 1)
                        if not live:
                            quit_flag[j & 1] = 1
                    if first[j] or once:
                        break
                    again = yield from meet("or", raises[j] or not live)
                    if not again:
                        break
                    if quit_flag[j & 1]:
                        return
                yield None
                if live:
                    p_full[j & 1].arrive()
                    s_empty[j & 1].arrive()
                yield None
            if j > 0 and last[j - 1]:
                yield from alive(pv_done[(j - 1) & 1], (j - 1) >> 1)
                for _ in range(4):  # rows by sixteens
                    if whole[j - 1] and any(x != j - 1 for x in inv):
                        raise Fault(f"sums {inv} for the piece that ends at {j - 1}")
                    yield None
            if j < n and last[j]:
                yield from meet("sync")
                if second:
                    yield from meet("sync")
                if w < WRITERS and whole[j]:
                    inv[w] = j
                yield None
                if third:
                    yield from meet("sync")

    roles = {"issue": issue(), **{f"softmax {w}": softmax(w) for w in range(WARPS)}}
    state, quiet, snapshot = {}, 0, None
    while roles:
        name = rnd.choice(list(roles))
        expire = state.get(name) == "wait" and (quiet > 200 or (aborted[0] and rnd.random() < 0.05) or rnd.random() < early)
        try:
            state[name] = roles[name].send(expire) if name in state else next(roles[name])
        except StopIteration:
            del roles[name]
            state.pop(name, None)
        now = (tuple(sorted(state.items(), key=str)), meeting["generation"], len(meeting["here"]),
               sum(b.phase * 16 + b.left for bs in (s_full, s_empty, p_full, pv_done) for b in bs))
        quiet = quiet + 1 if now == snapshot else 0
        snapshot = now
        if quiet > 3000:
            raise Fault("held for good: " + ", ".join(f"{k} {v}" for k, v in state.items()))
    return not aborted[0]


def test_every_warp_ends_and_has_its_own_sums():
    clean = sum(simulate(seed) for seed in range(400))
    assert 40 < clean < 360


@pytest.mark.parametrize("without", ["third", "agree"])
def test_the_model_sees_what_each_rule_is_for(without):
    faults = 0
    for seed in range(150):
        try:
            simulate(seed, **{without: False})
        except Fault:
            faults += 1
    assert faults > 5


def test_the_sums_are_safe_behind_the_first_meeting():
    """A warp writes a piece's results before it comes to the next one's end; the second meeting is for what the sums are made of."""
    for seed in range(150):
        simulate(seed, second=False)
