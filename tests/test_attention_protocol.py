"""The waits of the tcgen05 attention kernel on the CPU: its roles (loaders, the
issuer of the products, two softmax groups) as the sequences of waits, arrivals
and stage uses that their code makes, under random schedules.  Every schedule
has to end, no role may use a stage that another still owns, and a wait by
parity has to mean the phase it was written for."""
import os
import random
import re

import pytest

import mixed_precision_quantized_quantize_b200 as q


class Barrier:
    def __init__(self, need):
        self.need, self.phase, self.count = need, 0, 0

    def arrive(self):
        self.count += 1
        assert self.count <= self.need
        if self.count == self.need:
            self.phase, self.count = self.phase + 1, 0

    def passed(self, index):
        """Whether the wait for phase `index` goes on.  By parity it could be mistaken
        for another only if that were two phases away."""
        assert self.phase in (index, index + 1), (self.phase, index)
        return self.phase > index


def simulate(n, stages, early, seed, last_waits=True):
    """n tiles; early: tiles that the loaders have in flight before the first handed
    over (fp16: two, quantised: the conversion waits itself, none).  last_waits: a group waits for the product before the last one before it goes on to the last."""
    rng = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(1) for _ in range(stages)]
    s_full = [[Barrier(1), Barrier(1)] for _ in range(2)]
    p_full = [[Barrier(1), Barrier(1)] for _ in range(2)]
    pv = [Barrier(1), Barrier(1)]
    holds = {}   # stage -> tile being read
    queue = []   # products in order: (what to do when they are done)

    def loaders():
        for t in range(n + early):
            if early and t >= early:
                yield lambda: True
                full[(t - early) % stages].arrive()
            if t < n:
                if t >= stages:
                    yield lambda t=t: empty[t % stages].passed(t // stages - 1)
                assert t % stages not in holds, "a stage is filled while it is read"
                holds[t % stages] = t
                if not early:
                    full[t % stages].arrive()
            yield lambda: True

    def score(t, g):
        if g == 0:
            yield lambda: full[t % stages].passed(t // stages)

        def done():
            assert holds[t % stages] == t
            s_full[g][t & 1].arrive()
        queue.append(done)

    def values(t, g):
        yield lambda: p_full[g][t & 1].passed(t >> 1)

        def done():
            assert holds[t % stages] == t
            pv[g].arrive()
            if g == 1:
                del holds[t % stages]
                empty[t % stages].arrive()
        queue.append(done)

    def issuer():
        for t in range(n + 1):
            for g in range(2):
                if t < n:
                    yield from score(t, g)
            for g in range(2):
                if t > 0:
                    yield from values(t - 1, g)

    def softmax(g):
        for t in range(n):
            yield lambda t=t: full[t % stages].passed(t // stages)
            yield lambda t=t: s_full[g][t & 1].passed(t >> 1)
            assert holds[t % stages] == t  # its scales and masks are still there
            # the maximum moves: O has to stand still (and at the last tile in any case)
            if t > 0 and (rng.random() < 0.5 or (t == n - 1 and last_waits)):
                yield lambda t=t: pv[g].passed(t - 1)
            p_full[g][t & 1].arrive()
        if n:
            yield lambda: pv[g].passed(n - 1)

    roles = {}
    for name, r in (("loaders", loaders()), ("issuer", issuer()), ("softmax 0", softmax(0)), ("softmax 1", softmax(1))):
        try:
            roles[name] = [r, next(r)]
        except StopIteration:
            pass
    while roles or queue:
        ready = [k for k, (_, c) in roles.items() if c()]
        moves = ready + (["product"] if queue else [])
        if not moves:
            return False  # nobody can go on
        k = rng.choice(moves)
        if k == "product":
            queue.pop(0)()
            continue
        try:
            roles[k][1] = next(roles[k][0])
        except StopIteration:
            del roles[k]
    assert not holds
    return True


@pytest.mark.parametrize("stages,early", [(4, 2), (3, 0)])  # fp16; INT8 and INT4
@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 5, 8, 13, 24])
def test_every_schedule_ends(stages, early, n):
    for seed in range(60):
        assert simulate(n, stages, early, seed)


def test_a_stuck_order_is_seen():
    """Two tiles in flight before the first is handed over, in one stage: stuck, and
    the model says so."""
    assert not any(simulate(24, 1, 2, seed) for seed in range(20))


def test_a_wait_for_the_wrong_phase_is_seen():
    """Without the wait at the last tile, the last wait may meet a barrier two phases
    behind, which its parity cannot tell from the right one."""
    with pytest.raises(AssertionError):
        for seed in range(60):
            simulate(8, 3, 0, seed, last_waits=False)


def test_a_warpgroup_meets_one_register_instruction():
    """setmaxnreg is for a whole warpgroup: all of its warps have to meet the same
    instruction, whatever their roles.  So there is one to take registers and one to
    give them back, before the roles part, and what is taken was there at the launch."""
    with open(os.path.join(os.path.dirname(q.LIB_PATH), "csrc", "tree_attention_wide.cu")) as f:
        text = f.read()
    code = re.sub(r"//[^\n]*", "", text)
    sites = [(m.start(), m.group(1), int(m.group(2)))
             for m in re.finditer(r"setmaxnreg\.(inc|dec)\.sync\.aligned\.u32 (\d+);", code)]
    assert [s[1] for s in sites] == ["inc", "dec"]
    roles = code.index("s_col(g, buf) + lanes")  # the first line that only one role runs
    assert all(s[0] < roles for s in sites) and code.rindex("if (warp", 0, roles) > sites[1][0]
    # two row blocks: 8 softmax warps, 6 loaders, one for the scales, one for the products
    blocks, loaders = 2, int(re.search(r"kLoaders = (\d+);", code).group(1))
    softmax, others = blocks * 128, loaders + 64
    assert softmax % 128 == 0 and others % 128 == 0  # whole warpgroups on either side
    at_launch = 65536 // (softmax + others)
    assert softmax * sites[0][2] + others * sites[1][2] <= (softmax + others) * at_launch


def run_out(n, stages, early, role, wait, seed):
    """The same roles when wait number `wait` of `role` never comes to its end.  Once nobody
    can go on, some role's wait runs out: it sets the CTA's abort flag, which all other
    waits look at.  Returns the groups that wrote results, or None where the stalled wait
    was never reached."""
    rng = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(1) for _ in range(stages)]
    s_full = [[Barrier(1), Barrier(1)] for _ in range(2)]
    p_full = [[Barrier(1), Barrier(1)] for _ in range(2)]
    pv, drain = [Barrier(1), Barrier(1)], Barrier(1)
    holds, queue, wrote = {}, [], []

    def loaders():
        for t in range(n + early):
            if early and t >= early:
                full[(t - early) % stages].arrive()
            if t < n:
                if t >= stages and not (yield lambda t=t: empty[t % stages].passed(t // stages - 1)):
                    break
                assert t % stages not in holds, "a stage is filled while it is read"
                holds[t % stages] = t
                if not early:
                    full[t % stages].arrive()

    def values(t):
        for g in range(2):
            if not (yield lambda g=g: p_full[g][t & 1].passed(t >> 1)):
                return False

            def done(g=g):
                assert holds[t % stages] == t
                pv[g].arrive()
                if g == 1:
                    del holds[t % stages]
                    empty[t % stages].arrive()
            queue.append(done)
        return True

    def issuer():
        alive = True
        for t in range(n):
            alive = yield lambda t=t: full[t % stages].passed(t // stages)
            if not alive:
                break
            for g in range(2):
                def done(t=t, g=g):
                    assert holds[t % stages] == t
                    s_full[g][t & 1].arrive()
                queue.append(done)
            if t > 0:
                alive = yield from values(t - 1)
            if not alive:
                break
        if alive and n > 0:
            yield from values(n - 1)
        # what was issued has to end before its memory is given back: this wait does not
        # look at the flag
        nonlocal draining
        draining = True
        queue.append(drain.arrive)
        assert (yield lambda: drain.passed(0))
        assert not queue

    def softmax(g):
        alive = True
        for t in range(n):
            alive = (yield lambda t=t: full[t % stages].passed(t // stages))
            alive = alive and (yield lambda t=t: s_full[g][t & 1].passed(t >> 1))
            if not alive:
                break
            if t > 0 and (rng.random() < 0.5 or t == n - 1):
                alive = yield lambda t=t: pv[g].passed(t - 1)
                if not alive:
                    break
            p_full[g][t & 1].arrive()
        if alive and n > 0:
            alive = yield lambda: pv[g].passed(n - 1)
        if alive:
            assert pv[g].phase == n  # every product is in
            wrote.append(g)

    roles, waits, reached, abort, draining = {}, {}, False, False, False

    def step(name, make):
        """Let a role go on; make(r): its next wait."""
        nonlocal reached
        r = roles[name][0]
        try:
            condition = make(r)
        except StopIteration:
            del roles[name]
            return
        waits[name] = waits.get(name, -1) + 1
        if name == role and waits[name] == wait and not (name == "issuer" and draining):
            reached = True
            condition = lambda: False  # noqa: E731
        roles[name][1] = condition

    for name, r in (("loaders", loaders()), ("issuer", issuer()), ("softmax 0", softmax(0)), ("softmax 1", softmax(1))):
        roles[name] = [r, None]
        step(name, next)
    while roles or queue:
        ready = [(k, True) for k, (_, c) in roles.items() if c()]
        if abort:
            ready += [(k, False) for k, (_, c) in roles.items() if not c() and not (k == "issuer" and draining)]
        moves = ready + ([("product", True)] if queue else [])
        if not moves:
            assert not abort, "a role waits on after the abort"
            abort = True  # a wait has run out
            continue
        k, ok = rng.choice(moves)
        if k == "product":
            queue.pop(0)()
        else:
            step(k, lambda r: r.send(ok))
    return wrote if reached else None


@pytest.mark.parametrize("stages,early", [(4, 2), (3, 0)])
@pytest.mark.parametrize("role", ["loaders", "issuer", "softmax 0", "softmax 1"])
def test_a_wait_that_runs_out_ends_every_role(stages, early, role):
    """Whichever wait stands still: every role ends, what was issued has ended before the
    memory goes back, and a group that writes its rows has all of its products."""
    met = 0
    for n in (1, 2, 3, 7, 12):
        for wait in range(3 * n + 1):
            for seed in range(6):
                wrote = run_out(n, stages, early, role, wait, seed)
                if wrote is not None:
                    met += 1
                    assert not (role.startswith("softmax") and int(role[-1]) in wrote)
    assert met > 50
