"""The hand-offs of linear attention's two tcgen05 kernels, model-checked on the CPU.

Each role (two actors where it is several warps, which may drift apart) is written as its waits,
arrivals and uses of shared places in the kernel's order, for every chunk of every value head that a
block walks.  Random schedules, with copies and products that complete at random later times, check

* no deadlock, and no parity aliasing: a wait for completion k never finds its barrier two phases on;
* no race: any two uses of a place, one of them a write, are ordered by what their actors have waited
  for (vector clocks), whatever order this schedule happened to take.

The models mirror gated_delta_rule_07_gb300/csrc/gdn_linear_tc.cu and must be kept in step with it.
Planted bugs have to be found, among them a head's start that does not wait for the weights' warps.
That a warpgroup's warps set their registers together is read from the kernels' source.
"""
import os
import random
import re

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.phase, self.clock, self.clocks = count, 0, 0, {}, []

    def arrive(self, n, clock):
        self.arrived += n
        assert self.arrived <= self.count, "over-arrival"
        join(self.clock, clock)
        if self.arrived == self.count:
            self.clocks.append(self.clock)
            self.arrived, self.clock, self.phase = 0, {}, self.phase + 1


def join(clock, other):
    for a, t in other.items():
        if clock.get(a, 0) < t:
            clock[a] = t


class Race(Exception):
    pass


class Places:
    """Who used a place last: how ('r', 'w', or 'u': an atomic update, unordered among its like)."""

    def __init__(self):
        self.uses = {}

    def use(self, who, clock, place, how):
        before = self.uses.setdefault(place, [])
        for b, t, h in before:
            if b != who and clock.get(b, 0) < t and not (h == how and how in "ru"):
                raise Race(f"RACE: {who} uses {place} ({how}) beside {b} ({h})")
        if how == "w":
            del before[:]
        before[:] = [u for u in before if u[0] != who or u[2] != how] + [(who, clock.get(who, 0), how)]


def run(roles, counts, seed, races=True, max_steps=100000):
    """Runs the roles' generators to their ends under a random schedule; what went wrong, or None.

    ('wait', bar, k)  ('test', bar, k): whether it has completed    ('arrive', bar, n)
    ('use', how, *places)    ('mma', reads, writes): in order    ('commit', bar)
    ('copy', bar, reads, writes): completes any time later, arriving at bar (or, for None, where
    ('copied',) waits for)"""
    rng = random.Random(seed)
    bars, places = {b: Bar(n) for b, n in counts.items()}, Places()
    if not races:
        places.use = lambda *_: None
    gens, ops, clocks = {n: g() for n, g in roles.items()}, {}, {n: {n: 1} for n in roles}
    products, copies, serial = [], [], [0]   # products: (clock, barriers); copies: (clock, bar)
    stored = {}

    def step(name, value=None):
        try:
            ops[name] = gens[name].send(value)
        except StopIteration:
            del ops[name]

    def launch(name, clock, reads, writes):
        serial[0] += 1
        who = f"async{serial[0]}"
        clock = {**clock, who: 1}
        for p in reads:
            places.use(who, clock, p, "r")
        for p in writes:
            places.use(who, clock, p, "w")
        return clock

    for n in roles:
        step(n)
    pipe = {}   # what the products so far have ordered
    try:
        for _ in range(max_steps):
            if not ops:
                return None
            ready = []
            for n, op in ops.items():
                if op[0] == "wait":
                    phase = bars[op[1]].phase
                    if phase >= op[2] + 2:
                        return f"ALIAS: {n} waits for {op[1]} {op[2]}, {phase} phases are done"
                    if phase == op[2] + 1:
                        ready.append(("role", n))
                elif op[0] != "copied" or not stored.get(n):
                    ready.append(("role", n))
            if products:
                ready.append(("product", None))
            ready += [("copy", i) for i in range(len(copies))]
            if not ready:
                return f"DEADLOCK: {ops}"
            kind, x = rng.choice(ready)
            if kind == "product":
                clock, at = products.pop(0)
                for b in at:
                    bars[b].arrive(1, clock)
            elif kind == "copy":
                clock, b, owner = copies.pop(x)
                if b is None:
                    stored[owner].remove(clock)
                    join(clocks[owner], clock)
                else:
                    bars[b].arrive(1, clock)
            else:
                op, clock, back = ops[x], clocks[x], None
                clock[x] += 1
                if op[0] == "wait":
                    join(clock, bars[op[1]].clocks[op[2]])
                elif op[0] == "test":
                    assert bars[op[1]].phase <= op[2] + 1
                    back = bars[op[1]].phase == op[2] + 1
                elif op[0] == "arrive":
                    bars[op[1]].arrive(op[2], clock)
                elif op[0] == "use":
                    for p in op[2:]:
                        places.use(x, clock, p, op[1])
                elif op[0] == "mma":
                    pipe = launch(x, {**pipe, **clock}, op[1], op[2])
                    products.append((pipe, []))
                elif op[0] == "commit":
                    if products:
                        products[-1][1].append(op[1])
                    else:
                        bars[op[1]].arrive(1, {**pipe, **clock})
                elif op[0] == "copy":
                    c = launch(x, dict(clock), op[2], op[3])
                    copies.append((c, op[1], x))
                    if op[1] is None:
                        stored.setdefault(x, []).append(c)
                step(x, back)
    except Race as e:
        return str(e)
    return "too many steps"


def W(bar, k):
    return "wait", bar, k


def A(bar, n):
    return "arrive", bar, n


def tile(name, stage, rows=(0, 1), cols=(0, 1)):
    return [f"{name}{stage}.{r}{c}" for r in rows for c in cols]


# ----------------------------------------------------------------------------- the pass
def linear_pass(chunks, share, state_waits=True, kept_until_read=True, whole=True):
    """chunks of a segment, share: value heads that the block walks one after another; whole: chunks of
    128 tokens, whose outputs leave by TMA.  state_waits: a head's start waits for the weights' warps to
    have begun the one before; kept_until_read: a row's exponent stays until the outputs were scaled."""
    total = chunks * share

    def bar(name, it):
        return f"{name}{it & 1}"

    def loader():
        loaded = 0
        for it in range(-2, total):
            more = loaded < total
            if more:
                if it >= 0:
                    yield W(bar("Free", it), it >> 1)
                yield "copy", bar("Full", it), [], tile("Z", it & 1) + tile("X", it & 1)
            if it >= 0:
                yield W(bar("Out", it), it >> 1)
                if it // chunks + 1 == share and whole:
                    yield "copy", None, tile("Y", it & 1), []
                    if more:
                        yield "copied",
            if more:
                yield "copy", bar("FullY", it), [], tile("Y", it & 1)
                loaded += 1
        yield "copied",

    def mma():
        grown = scored = c = 0
        for turn in range(-1, 2 * total):
            it, odd = turn >> 1, turn & 1
            if turn >= 0 and not odd:
                yield W(bar("Values", it), it >> 1)
                if c + 1 < chunks:
                    if grown:
                        yield W("Taken", grown - 1)
                    yield "mma", tile("X", it & 1) + tile("Y", it & 1), ["G.0", "G.1"]
                    yield "commit", "Grown"
                    grown += 1
            elif turn >= 0:
                yield W(bar("Weights", it), it >> 1)
                if it > 0:
                    yield W(bar("SumsRead", it - 1), (it - 1) >> 1)
                yield "mma", [f"W{it & 1}.0", f"W{it & 1}.1"] + tile("Y", it & 1), ["O.0", "O.1"]
                yield W(bar("Targets", it), it >> 1)
                yield W("StateIn", it)
                yield "mma", [f"z{it & 1}.0", f"z{it & 1}.1", "S.0", "S.1"], ["O.0", "O.1"]
                yield "commit", "Sums"
                yield "commit", bar("Free", it)
                c = (c + 1) % chunks
            if scored < total and scored <= it + 1:
                there = odd or (yield "test", bar("Full", scored), scored >> 1)
                if there:
                    s = scored & 1
                    yield W(bar("Full", scored), scored >> 1)
                    yield "mma", tile("Z", s) + tile("X", s), [f"W{s}.0", f"W{s}.1", f"z{s}.0", f"z{s}.1"]
                    yield "commit", bar("Scores", scored)
                    scored += 1

    def weights(h):
        def role():
            it = 0
            for g in range(share):
                yield W("Start", g)
                yield "use", "r", f"max{g & 1}"
                yield A("named", 64)
                yield W("named", 2 * g)
                if h == 0:
                    yield "use", "w", f"max{~g & 1}"
                yield "use", "w", f"powers.{h}"
                yield A("named", 64)
                yield W("named", 2 * g + 1)
                if state_waits:
                    yield A("Begun", 64)
                yield "use", "r", "powers.0", "powers.1"
                for _ in range(chunks):
                    s = it & 1
                    yield W(bar("Rows", it), it >> 1)
                    yield W(bar("Scores", it), it >> 1)
                    yield "use", "r", f"e{s}.{h}", "powers.0", "powers.1", f"W{s}.{h}", f"z{s}.{h}"
                    yield "use", "w", f"W{s}.{h}"
                    yield A(bar("Weights", it), 64)
                    yield "use", "r", *tile("Z", s, rows=(h,))
                    yield "use", "w", f"z{s}.{h}"
                    yield A(bar("Targets", it), 64)
                    it += 1
        return role

    def state(h):
        def give(it, g):
            s = it & 1
            yield "use", "r", f"e{s}.0", f"e{s}.1", f"O.{h}"
            yield A(bar("SumsRead", it), 128)
            if g + 1 == share and whole:
                yield "use", "w", *tile("Y", s, cols=(h,))
            yield A(bar("Out", it), 128)

        def role():
            grown = 0
            for it in range(total + 1):
                g, c = divmod(it, chunks)
                if it < total and c == 0:
                    if g > 0 and state_waits:
                        yield W("Begun", g - 1)
                    yield "use", "u", f"max{g & 1}"
                    yield A("Start", 128)
                    yield W("Start", g)
                    yield "use", "r", f"max{g & 1}"
                if it > 0:
                    yield W("Sums", it - 1)
                    yield from give(it - 1, (it - 1) // chunks)
                if it < total:
                    yield "use", "w", f"S.{h}"
                    yield A("StateIn", 128)
                    if c + 1 < chunks:
                        yield W("Grown", grown)
                        yield "use", "r", f"G.{h}"
                        yield A("Taken", 128)
                        grown += 1
        return role

    def opener(h):
        def role():
            it = 0
            for _ in range(share):
                for c in range(chunks):
                    s = it & 1
                    yield W(bar("Full", it), it >> 1)
                    yield "use", "r", *tile("Z", s, rows=(h,))
                    if it >= 2 and kept_until_read:
                        yield W(bar("SumsRead", it - 2), (it - 2) >> 1)
                    yield "use", "w", f"e{s}.{h}"
                    yield A(bar("Rows", it), 64)
                    if c + 1 < chunks:
                        yield W(bar("Scores", it), it >> 1)
                        yield "use", "w", *tile("X", s, rows=(h,))
                    yield W(bar("FullY", it), it >> 1)
                    yield "use", "w", *tile("Y", s, rows=(h,))
                    yield A(bar("Values", it), 64)
                    it += 1
        return role

    roles = dict(loader=loader, mma=mma)
    for h in (0, 1):
        roles.update({f"weights{h}": weights(h), f"state{h}": state(h), f"open{h}": opener(h)})
    counts = dict(StateIn=256, Grown=1, Taken=256, Sums=1, Start=256, Begun=128, named=128)
    for i in (0, 1):
        counts.update({f"{n}{i}": k for n, k in dict(
            Full=1, FullY=1, Scores=1, Free=1, Values=128, Weights=128, Rows=128, Targets=128,
            SumsRead=256, Out=256).items()})
    return roles, counts


# ----------------------------------------------------------------------------- a segment's own state
def linear_state(tiles, parts_kept=True):
    """tiles of 64 tokens; parts_kept: the parts' columns are written when the products that read them
    two tiles ago are done."""
    stages = 5

    def loader():
        for i in range(tiles):
            if i >= stages:
                yield W(f"Free{i % stages}", i // stages - 1)
            yield "copy", f"Full{i % stages}", [], tile("X", i % stages) + tile("Y", i % stages)

    def mma():
        for i in range(tiles):
            b = i & 1
            yield W(f"Ready{b}", i >> 1)
            if i >= 2:
                yield W(f"Taken{b}", (i >> 1) - 1)
            yield "mma", tile("X", i % stages) + [f"parts{b}.0", f"parts{b}.1"], [f"D{b}.0", f"D{b}.1"]
            yield "commit", f"Done{b}"
            yield "commit", f"Free{i % stages}"

    def split(h):
        def role():
            for i in range(tiles):
                b, s = i & 1, i % stages
                yield W(f"Full{s}", i // stages)
                if i >= 2 and parts_kept:
                    yield W(f"Done{b}", (i >> 1) - 1)
                yield "use", "r", *tile("Y", s)
                yield "use", "w", f"parts{b}.{h}", *tile("X", s, rows=(h,))
                yield A(f"Ready{b}", 256)
            yield "use", "u", "top"
            yield A("all", 1)
        return role

    def add(h):
        def role():
            for i in range(tiles):
                b = i & 1
                yield W(f"Done{b}", i >> 1)
                yield "use", "r", f"D{b}.{h}"
                yield A(f"Taken{b}", 128)
            yield A("all", 1)
        return role

    def end():
        yield W("all", 0)
        yield "use", "r", "top"

    roles = dict(loader=loader, mma=mma, end=end)
    for h in (0, 1):
        roles.update({f"split{h}": split(h), f"add{h}": add(h)})
    counts = {"all": 4}
    counts.update({f"{n}{i}": 1 for n in ("Full", "Free") for i in range(stages)})
    for i in (0, 1):
        counts.update({f"Ready{i}": 512, f"Done{i}": 1, f"Taken{i}": 256})
    return roles, counts


def check(make, trials=150):
    for seed in range(trials):
        wrong = run(*make(), seed)
        if wrong:
            return wrong
    return None


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("share", [1, 2, 3, 4])
@pytest.mark.parametrize("chunks", [1, 2, 3])
def test_the_pass(chunks, share, whole):
    assert check(lambda: linear_pass(chunks, share, whole=whole)) is None


@pytest.mark.parametrize("tiles", [1, 2, 3, 6, 12])
def test_the_states(tiles):
    assert check(lambda: linear_state(tiles)) is None


@pytest.mark.parametrize("share", [2, 3, 4])
def test_a_heads_start_that_does_not_wait_is_found(share):
    """One chunk a head: nothing else that the state waits for says that the weights' warps have begun
    the head before.  The maximum that they clear can be the next head's, or their wait be passed by."""
    planted = [linear_pass(1, share, state_waits=False) for _ in range(300)]
    wrong = [run(*p, seed) for seed, p in enumerate(planted)]
    assert any(w and "RACE" in w and "max" in w for w in wrong)
    wrong = [run(*p, seed, races=False) for seed, p in enumerate(planted)]
    assert any(w and "ALIAS" in w and "Start" in w for w in wrong)


def test_other_planted_bugs_are_found():
    wrong = check(lambda: linear_pass(2, 2, kept_until_read=False), 400)
    assert wrong and "RACE" in wrong and " e" in wrong
    wrong = check(lambda: linear_state(4, parts_kept=False), 400)
    assert wrong and "RACE" in wrong and "parts" in wrong


# ----------------------------------------------------------------------------- registers
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "gated_delta_rule_07_gb300", "csrc", "gdn_linear_tc.cu")


@pytest.mark.parametrize("kernel,threads", [("linear_state_tc_kernel", "kStateThreads"),
                                            ("linear_pass_tc_kernel", "kPassThreads")])
def test_a_warpgroup_sets_its_registers_at_one_place(kernel, threads):
    """setmaxnreg is for all warps of a warpgroup together: each of them has to come to the same one,
    which stands first under the branches of the roles, and the registers have to add up."""
    with open(SOURCE) as f:
        text = f.read()
    known = {}
    for line in re.findall(r"constexpr int ([^;]*);", text):
        for name, value in re.findall(r"(k\w+) = ([^,]+)", line):
            try:
                known[name] = int(eval(value.replace("/", "//"), {}, known))
            except (NameError, SyntaxError):
                pass
    body = text[text.index(f"\n{kernel}("):]
    body = body[:body.index("\n}\n")].split("\n")
    branches = []   # [condition, registers of the call under it] of the first `if (warp ...)` chain
    for i, line in enumerate(body):
        role = re.match(r"  (?:} else )?if \((warp [<>=].*)\) {", line)
        if role:
            condition = role.group(1)
        elif line.startswith("  } else {") and branches:
            condition = "True"
        else:
            continue
        after = next(x for x in body[i + 1:] if x.strip() and not x.strip().startswith("//"))
        call = re.match(r"    (?:take|leave)_registers<(\d+)>\(\);", after)
        if call:
            branches.append((condition.replace("/", "//"), int(call.group(1))))
    calls = sum(len(re.findall(r"(?:take|leave)_registers<", line)) for line in body)
    assert len(branches) >= 3 and calls == len(branches)

    def place(warp):
        return next(i for i, (c, _) in enumerate(branches) if eval(c, {}, {**known, "warp": warp}))

    warps = known[threads] // 32
    groups = [{place(w) for w in range(g, g + 4)} for g in range(0, warps, 4)]
    assert warps % 4 == 0 and all(len(g) == 1 for g in groups), groups
    at_launch = 65536 // known[threads] // 8 * 8
    assert sum(branches[p][1] for g in groups for p in g) <= at_launch * warps // 4
