"""The ring of units in the pair kernel's shared memory: its scheduler may write a unit into
a slot only when every role has read the unit that was there, whatever the warps' speeds.

The roles' program orders and the waits between them make a partial order of their steps; the
rule by which the scheduler waits is taken from the source."""

import itertools
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "sparse_mla_decode_csr_gb300", "csrc", "smla_paged_attend.cu")


def ring_size():
    return int(re.search(r"constexpr int kJobs = (\d+);", open(SOURCE).read()).group(1))


def waited_for(n):
    """Units that the softmax warps are through with before the scheduler hands out unit n."""
    k_jobs, units = ring_size(), []

    def wait(slot_of):
        units.append(slot_of - k_jobs)
        return True

    rule = re.search(r"if \(n >= kJobs\) fine = (.*?);", open(SOURCE).read()).group(1)
    if n >= k_jobs:
        eval(rule.replace("&&", "and").replace("||", "or"), {"n": n, "kJobs": k_jobs, "wait": wait})
    return units


class Order:
    """Steps and what each comes after; `before` of a step is a bit set of all steps that do."""

    def __init__(self):
        self.after = {}

    def add(self, step, *earlier):
        self.after.setdefault(step, []).extend(e for e in earlier if e is not None)

    def solve(self):
        """Raises when steps wait for each other in a circle."""
        self.index = {s: i for i, s in enumerate(self.after)}
        self.before, state = {}, {}
        for root in self.after:
            stack = [(root, iter(self.after[root]))]
            if state.get(root) == 2:
                continue
            state[root] = 1
            while stack:
                step, rest = stack[-1]
                nxt = next((e for e in rest if state.get(e) != 2), None)
                if nxt is not None:
                    assert nxt in self.after, f"{step} waits for {nxt}, which never happens"
                    assert state.get(nxt) != 1, f"{step} and {nxt} wait for each other"
                    state[nxt] = 1
                    stack.append((nxt, iter(self.after[nxt])))
                    continue
                bits = 0
                for e in self.after[step]:
                    bits |= self.before[e] | 1 << self.index[e]
                self.before[step] = bits
                state[step] = 2
                stack.pop()
        return self

    def comes_before(self, a, b):
        return bool(self.before[b] >> self.index[a] & 1)


def order_of(tiles):
    """The steps of a worker whose units have so many key tiles."""
    o, k_jobs = Order(), ring_size()
    unit_of = [u for u, n in enumerate(tiles) for _ in range(n)]
    ends = [u + 1 == len(unit_of) or unit_of[u + 1] != unit_of[u] for u in range(len(unit_of))]
    total, last = len(unit_of), len(tiles)  # unit `last`: there is no more
    at = lambda g: unit_of[g] if g < total else last
    for n in range(last + 1):
        o.add(("publish", n), ("publish", n - 1) if n else None, *(("free", u) for u in waited_for(n)))
    # a loader group's tiles are every other one; it reads the units of the two tiles behind
    # the one in hand before it stores that
    for group in (0, 1):
        prev = None

        def read(upto, prev):
            # (the units' records are read one after the other as the cursor goes over their ends)
            seen = read.seen
            while seen <= min(upto, last):
                o.add(("read", ("loaders", group), seen), ("publish", seen), prev)
                prev = ("read", ("loaders", group), seen)
                seen += 1
            read.seen = seen
            return prev

        read.seen = 0
        prev = read(0, prev)
        if group == 1:
            prev = read(at(1), prev)
        for g in range(group, total, 2):
            if g == 0 or unit_of[g - 1] != unit_of[g]:  # q, from the unit's record, behind the last QK
                step = ("again", group, g)
                o.add(step, prev, ("qk", g - 1) if g else None)
                prev = step
            prev = read(at(g + 1), prev)
            prev = read(at(g + 2), prev)
            step = ("store", g)
            o.add(step, prev, ("qk", g - 2) if g >= 2 else None, ("copied", g - 2) if g >= 2 else None)
            prev = step
    # the other roles read a unit, then do its tiles
    prev = {role: None for role in ("qk", "pv", "copier", "softmax")}
    for g in range(total):
        u = unit_of[g]
        for role in prev:
            if g == 0 or unit_of[g - 1] != u:
                o.add(("read", role, u), ("publish", u), prev[role])
                prev[role] = ("read", role, u)
        o.add(("qk", g), prev["qk"], ("store", g), ("scores", g - 2) if g >= 2 else None)
        o.add(("copied", g), prev["copier"], ("store", g), ("pv", g - 2) if g >= 2 else None)
        o.add(("scores", g), prev["softmax"], ("qk", g))  # S is read
        o.add(("p", g), ("scores", g), ("pv", g - 1) if g else None)
        o.add(("pv", g), prev["pv"], ("copied", g), ("p", g))
        prev.update(qk=("qk", g), copier=("copied", g), pv=("pv", g), softmax=("p", g))
        if ends[g]:
            o.add(("free", u), ("p", g), ("pv", g))
            prev["softmax"] = ("free", u)
    return o.solve(), k_jobs


def check(tiles):
    o, k_jobs = order_of(tiles)
    for n in range(k_jobs, len(tiles) + 1):
        for step in o.after:
            mine = (step[0] == "read" and step[2] == n - k_jobs) or (
                step[0] == "again" and sum(tiles[:n - k_jobs]) == step[2])
            if mine:
                assert o.comes_before(step, ("publish", n)), f"unit {n} may overwrite unit {n - k_jobs} before {step}: {tiles}"


def test_the_rule_is_found():
    assert ring_size() >= 2 and [waited_for(n) for n in range(ring_size())] == [[]] * ring_size()
    for n in range(ring_size(), 3 * ring_size()):
        assert n - ring_size() in waited_for(n)


@pytest.mark.parametrize("units", range(1, 8))
def test_no_unit_is_overwritten_before_every_role_has_read_it(units):
    for tiles in itertools.product((1, 2, 3) if units < 7 else (1, 2), repeat=units):
        check(tiles)


def test_units_drawn_at_random():
    r = random.Random(3)
    for _ in range(60):
        check([r.choice((1, 1, 1, 2, 3, 7)) for _ in range(r.randint(8, 40))])
