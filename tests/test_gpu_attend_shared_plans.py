"""Plans that csa2_attend_shared is given: heads that do not begin where they
say, in plans that the tile kernel makes itself and in those of a launch of
their own."""
import random

import pytest
import torch

from test_gpu_attend_shared import Case

pytestmark = pytest.mark.gpu


def valid_places(head):
    """Whether each place's head is where the run of equal heads around it begins."""
    ok, run = [], 0
    for k, h in enumerate(head):
        if k == 0 or h != head[k - 1]:
            run = k
        ok.append(h == run)
    return ok


def check_plan(c, head, shared):
    """c's queries at places 0 .. n - 1: those at valid places as the plan says,
    the others' outputs left as they were and the fault recorded."""
    n = len(head)
    ok = valid_places(head)
    c.order, c.head, c.shared = list(range(n)), list(head), list(shared)
    c.plan()
    c.out.fill_(77)
    c.lse.fill_(77)
    c.run(flags=0 if all(ok) else c.b.FLAG_BAD_QUERY)
    skipped = [k for k in range(n) if not ok[k]]
    assert (c.out[skipped] == 77).all() and (c.lse[skipped] == 77).all()
    # (what a skipped place's head names is not asked for)
    c.head = [h if good else k for k, (h, good) in enumerate(zip(head, ok))]
    c.check(only=[k for k in range(n) if ok[k]])


BAD_HEADS = [
    [0, 1, 0, 3, 4, 5],          # an even and an odd offset across another group
    [0, 1, 2, 0, 4, 5],
    [0, 0, 0, 1, 4, 4],          # a head that heads no group
    [0, 0, 0, 0, 1, 5],
    [0, 1, 0, 0, 0, 5],          # the neighbour agrees, the group is still not where it says
    [0, 0, 2, 3, 2, 2],
    [3, -4, 0, 2, 4, 99],        # behind, below, above
    [-1, -1, -1, 3, -(1 << 31), (1 << 31) - 1],
    [1, 1, 1, 1, 1, 1],          # a run that does not begin at its head
    [0, 0, 0, 3, 3, 3],          # none
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("head", BAD_HEADS)
def test_places_whose_group_begins_elsewhere(fmt, head):
    # unrelated sequences with lengths that every head's place asks for: a wrong first query shows
    c = Case([(0, [130 + 17 * i for i in range(6)])], fmt=fmt, page=16, seed=101)
    check_plan(c, head, [32 + 16 * i for i in range(6)])


@pytest.mark.parametrize("head", BAD_HEADS)
@pytest.mark.parametrize("before", [28, 31, 59, 90, 93, 170, 1022, 1500])
def test_such_places_behind_others(head, before):
    # across the warps and shares that look at the heads; up to 96 places and more
    lens = [20 + 3 * i for i in range(40)]
    n = before + 6
    c = Case([(0, lens)], page=16, queries=[(i % 40, lens[i % 40] - 1) for i in range(n)], seed=102)
    heads = [k - k % 5 for k in range(before)] + [h + before if -1 <= h < 99 else h for h in head]
    shared = [0] * before + [16] * 6
    ok = valid_places(heads)
    c.order, c.head, c.shared = list(range(n)), heads, shared
    c.plan()
    c.out.fill_(77)
    c.lse.fill_(77)
    c.run(flags=0 if all(ok) else c.b.FLAG_BAD_QUERY)
    for k in range(n):
        assert bool((c.out[k] == 77).all()) == (not ok[k]), k
        assert bool((c.lse[k] == 77).all()) == (not ok[k]), k
    c.head = [h if good else k for k, (h, good) in enumerate(zip(heads, ok))]
    c.check(only=[k for k in [0, 1, 4, *range(before - 3, n)] if ok[k]])


def test_one_run_over_many_shares():
    # one group of all places, its head far before the shares that look for it
    lens = [40 + i % 50 for i in range(60)]
    n = 2600
    c = Case([(2, lens)], page=16, queries=[(i % 60, lens[i % 60] - 1) for i in range(n)], seed=103)
    c.order, c.head, c.shared = list(range(n)), [0] * n, [32] + [0] * (n - 1)
    c.plan()
    c.run().check(only=[0, 1, 2, 3, 1023, 1024, 1025, 2598, 2599])


# ---------------------------------------------------------------- padded batches

def padded(n, live, page=16, fmt="bf16", seed=0):
    """n queries of which those of `live` have sequences: places group by group, padding a place each, mixed."""
    rng = random.Random(seed)
    lens = [64 + rng.randint(1, 400) for _ in range(9)]
    at = sorted(rng.sample(range(n), live))
    queries = [(-1, rng.choice([-1, 5]))] * n
    for j, i in enumerate(at):
        queries[i] = (j % 9, lens[j % 9] - 1 - (j // 9) % 30)
    return Case([(4, lens)], page=page, fmt=fmt, queries=queries, seed=seed), at


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n,live", [(1, 0), (2, 1), (16, 3), (64, 5), (76, 0), (90, 7), (96, 2), (97, 0), (300, 11), (2100, 9)])
def test_padded_batches(fmt, n, live):
    c, at = padded(n, live, fmt=fmt, seed=n)
    c.run().check(only=at)
    rest = [i for i in range(n) if i not in at]
    assert (c.out[rest] == 77).all() and (c.lse[rest] == 77).all()


def test_padding_inside_groups():
    # two empty places that would be a unit, one beside a query, one as the head
    lens = [70, 90, 110, 130]
    c = Case([(4, lens)], page=16, queries=[(0, 69), (-1, 3), (-1, 4), (1, 89), (-1, 5), (2, 109), (3, 129)], seed=104)
    c.order, c.head, c.shared = [0, 3, 1, 2, 4, 5, 6], [0] * 7, [64] + [0] * 6
    c.plan()
    c.run().check(only=[0, 3, 5, 6])
    assert (c.out[[1, 2, 4]] == 77).all()


def test_places_without_a_query_cost_no_tile():
    # as many places, one row each: without a query they take well under half of the time
    n = 4096
    empty = Case([(0, [5])], page=16, queries=[(-1, 0)] * (n - 4) + [(0, 4)] * 4, seed=105)
    one = Case([(0, [5])], page=16, queries=[(0, 0)] * n, seed=105)
    best = {}
    for name, c in (("one", one), ("empty", empty)):
        call = c.call()
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                call.run()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best[name] = min(times[1:])
    assert best["empty"] < 0.5 * best["one"], best
