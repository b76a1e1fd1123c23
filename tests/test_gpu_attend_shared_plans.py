"""csa2_attend_shared: plans whose heads do not begin where they say, in plans
that the tile kernel makes itself and in those of a launch of their own; padded
batches; its outputs beside csa2_attend_paged's, the flags of lengths that are
cut, positions far past the table, very many queries."""
import random

import pytest
import torch

from paged_common import DIM, HEADS, U16, U32, attend_one, layer_turned, page_values
from test_gpu_attend_shared import DEV, Case

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


# ---------------------------------------------------------------- results

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_outputs_of_both_attentions_on_the_same_queries(fmt):
    """Groups found by csa2_query_groups; csa2_attend_paged's out and lse and
    csa2_attend_shared's, each within the bounds of the exact result, and so
    within twice them of each other."""
    c = Case([(7, [16 * 7 + 30, 16 * 7 + 9, 16 * 7 + 77]), (5, [16 * 5 + 3, 16 * 5 + 40]), (0, [90])], fmt=fmt, page=16, per=2, seed=106)
    n = len(c.seq)
    order, head = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
    shared = torch.empty(n, dtype=torch.int64, device=DEV)
    c.ctx.query_groups(c.table, 16, c.codes.shape[0], c.pos_d, c.seq_d, 40, order, head, shared)
    c.order, c.head, c.shared = order.tolist(), head.tolist(), shared.tolist()
    assert c.shared[0] == 16 * 7 and c.shared[6] == 16 * 5
    c.plan()
    c.run().check()
    one, one_lse = c.out.clone(), c.lse.clone()
    ws = c.b.workspace(c.ctx.attend_paged_workspace_size(n), DEV)
    c.out.fill_(77)
    c.lse.fill_(77)
    c.ctx.attend_paged(c.kv, c.q, c.pos_d, c.seq_d, c.out, ws, sink=c.sink, lse=c.lse)
    assert c.ctx.check()[0] == 0
    c.check()
    v, views = page_values(c.codes, c.scales, c.fmt), c.views()
    for i in range(n):
        _, _, bo, bl = attend_one(v, views[i], 16, c.q[i], c.pos[i], 0, 0, 0, c.sink, c.ctx.cfg)
        assert ((one[i] - c.out[i]).double().cpu().abs() <= 2 * bo).all()
        assert ((one_lse[i] - c.lse[i]).double().cpu().abs() <= 2 * bl).all()


@pytest.mark.parametrize("shared,missing", [(-(1 << 62), False), (-3, False), (0, False), (7, False), (16, False), (40, False), (64, False),
                                            (1000, True), (1 << 40, True), ((1 << 63) - 1, True)])
def test_flags_of_lengths_that_are_cut(shared, missing):
    # the first query's sequence has 60 rows in four pages: of a common length past them the fourth's rows are its own,
    # the pages behind, which only the others see, missing
    c = Case([(3, [60, 70, 90])], page=16, seed=107)
    c.shared[0] = shared
    c.plan()
    c.run(flags=c.b.FLAG_BAD_PAGE if missing else 0)
    c.shared[0] = min(max(shared, 0), 16 * len(c.table_rows[0]))
    c.check()


def test_a_position_far_past_the_table():
    # every row of the table, rotated at 2^40
    t = 1 << 40
    c = Case([(2, [48, 48])], page=16, queries=[(0, 47), (1, t)], seed=108)
    c.run(flags=c.b.FLAG_BAD_PAGE).check(only=[0])
    cfg, row = c.ctx.cfg, c.views()[1]
    rows = page_values(c.codes, c.scales, c.fmt)[row].reshape(-1, DIM)
    tau, r = float(cfg.softmax_scale), int(cfg.rope_dim)
    q = layer_turned(c.q[1].double().cpu(), t, cfg)
    z = q @ rows.T * tau
    lse = torch.logsumexp(torch.cat((z, c.sink.double().cpu()[:, None]), -1), -1)
    w = torch.exp(z - lse[:, None])
    o = w @ rows
    # attend_one's bounds, and the angles: t f, f at most 1, is off by 2^-53 of itself in each double product and by
    # 2^-51 for frequencies two steps apart, on both sides below 2^-50 of 2^40: 2^-10 radians, which move a pair by as
    # much of its length, scores by tau times the pairs' lengths' products, and o as other errors of scores do
    turn = 2.0 ** -10
    pairs = lambda x: x[:, DIM - r:].reshape(x.shape[0], -1, 2).norm(dim=-1)  # noqa: E731
    mag, rope = tau * (q.abs() @ rows.abs().T), tau * (q[:, DIM - r:].abs() @ rows[:, DIM - r:].abs().T)
    delta = 40 * U32 * mag + (U16 ** 2 + 4 * U32) * rope + 2.0 ** -21 + turn * tau * (pairs(q) @ pairs(rows).T)
    # exp(delta) - 1 <= 1.1 delta, in numerator and denominator
    assert float(delta.max()) < 0.15
    S = torch.einsum("hn,hnd->hd", w * 1.1 * delta, (rows[None] - o[:, None]).abs()) * 1.1
    bound = (U16 + (len(rows) / 16 + 160) * U32) * (w @ rows.abs()) + S
    both = bound[:, DIM - r:].reshape(HEADS, -1, 2).sum(-1, keepdim=True).expand(-1, -1, 2).reshape(HEADS, r)
    length = (1 + turn) * turn * pairs(o)[:, :, None].expand(-1, -1, 2).reshape(HEADS, r)
    bound = torch.cat((bound[:, :DIM - r], both + length), -1)
    o = layer_turned(o, -float(t), cfg)
    bound = bound + U16 * (o.abs() + bound) + 1e-30
    assert ((c.out[1].double().cpu() - o).abs() <= bound).all()
    assert ((c.lse[1].double().cpu() - lse).abs() <= 1.1 * delta.amax(-1) + 8 * U32 * (1 + lse.abs())).all()


def test_very_many_queries():
    # a share of many places a thread in the plan
    n, lens = 40000, [3 + 7 * i for i in range(11)]
    rng = random.Random(109)
    c = Case([(0, lens)], page=16, queries=[(i % 11, rng.randint(0, lens[i % 11] - 1)) for i in range(n)], seed=109)
    at = [0, 1, 39, 40, 41, n - 2, n - 1] + rng.sample(range(n), 25)
    c.run().check(only=at)
    assert torch.isfinite(c.out).all() and torch.isfinite(c.lse).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("n", [4, 9, 10, 11, 12, 13, 18, 19, 20, 37, 38, 39])
def test_numbers_of_queries_around_the_joins(fmt, n):
    # every query split: of one prefix, and of sequences of their own
    Case([(40, [40 * 64 + 1 + 11 * i for i in range(n)])], fmt=fmt, page=64, seed=n).run().check(only=[0, n // 2, n - 1])
    Case([(0, [1300 + 11 * i for i in range(n)])], fmt=fmt, page=64, seed=n + 50).run().check(only=[0, n // 2, n - 1])
