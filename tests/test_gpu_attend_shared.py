"""csa2_attend_shared against a plain 64-bit form (paged_common.attend_one on
each query's own view of the table: the columns of its group's common beginning
from the group's first query, the others its own), at the sizes, groups,
formats, masks and streams where it can go wrong. Bounds as derived there: the
kernel's arithmetic is csa2_attend_paged's (rope channels as hi + lo, weights
rounded to bf16 for the products, fp32 sums joined from at most 76 partials)."""
import math
import random

import pytest
import torch

from gpu_common import context, require_gpu
from paged_common import DIM, FMT_NAMES, HEADS, U32, check_attend, page_values, random_pages

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """Sequences in groups, forks of one beginning each. groups: for each group
    (shared whole pages, [lengths]); a query at the last `per` positions of
    every sequence, or `queries` (sequence, position). Places group by group."""

    def __init__(self, groups, fmt="bf16", page=16, per=1, sink=True, seed=0, spare=2, rope=True, layers=0, extra_cols=0,
                 q_scale=1.0, queries=None, shuffle=False):
        from compressed_sparse_attention_gb300 import binding
        require_gpu()
        self.b = binding
        self.ctx = context(kv_format=fmt, **({} if rope else {"rope_dim": 0}))
        self.fmt, self.page = FMT_NAMES[fmt], page
        rng = random.Random(seed)
        n_pages = sum(w + sum(max(0, -(-n // page) - w) for n in lens) for w, lens in groups) + spare
        order = list(range(n_pages))
        rng.shuffle(order)
        rows, group_of_seq, self.lens = [], [], []
        for g, (whole, lens) in enumerate(groups):
            first = [order.pop() for _ in range(whole)]
            for n in lens:
                k = -(-n // page)
                rows.append(first[:k] + [order.pop() for _ in range(max(0, k - whole))])
                group_of_seq.append(g)
                self.lens.append(n)
        width = max(1, max(len(r) for r in rows))
        self.table_rows = [r + [-1] * (width - len(r)) for r in rows]
        self.codes, self.scales = random_pages(self.fmt, n_pages, page, seed, DEV, (layers,) if layers else ())
        if layers:
            self.codes = self.codes.transpose(0, 1).contiguous()[:, -1]
            self.scales = None if self.scales is None else self.scales.transpose(0, 1).contiguous()[:, -1]
        full = torch.full((len(rows), width + extra_cols), 7, dtype=torch.int32)
        full[:, :width] = torch.tensor(self.table_rows, dtype=torch.int32)
        self.table = full.to(DEV)[:, :width]
        queries = queries if queries is not None else [(b, n - per + i) for b, n in enumerate(self.lens) for i in range(per)]
        n = len(queries)
        if shuffle:
            rng.shuffle(queries)
        self.seq, self.pos = [b for b, _ in queries], [t for _, t in queries]
        # places: the queries of a group one after another
        self.order, self.head, self.shared = [], [], []
        for g, (whole, _) in enumerate(groups):
            mine = [i for i, b in enumerate(self.seq) if 0 <= b < len(group_of_seq) and group_of_seq[b] == g]
            for j, i in enumerate(mine):
                self.head.append(len(self.order) - j)
                self.order.append(i)
                self.shared.append(whole * page if j == 0 else 0)
        for i in range(n):
            if i not in self.order:  # queries without a sequence: a place of their own
                self.head.append(len(self.order))
                self.order.append(i)
                self.shared.append(0)
        gen = torch.Generator().manual_seed(seed + 1)
        self.q = (q_scale * torch.randn((n, HEADS, DIM), generator=gen)).to(torch.bfloat16).to(DEV)
        self.sink = torch.randn((HEADS,), generator=gen).to(DEV) if sink is True else sink
        self.seq_d = torch.tensor(self.seq, dtype=torch.int32, device=DEV)
        self.pos_d = torch.tensor(self.pos, dtype=torch.int64, device=DEV)
        self.out = torch.full((n, HEADS, DIM), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((n, HEADS), 77.0, device=DEV)
        self.ws = binding.workspace(self.ctx.attend_shared_workspace_size(max(n, 1)), DEV)
        self.kv = self.ctx.paged_kv(self.codes, self.table, self.scales)
        self.plan()

    def plan(self):
        self.order_d = torch.tensor(self.order, dtype=torch.int32, device=DEV)
        self.head_d = torch.tensor(self.head, dtype=torch.int32, device=DEV)
        self.shared_d = torch.tensor(self.shared, dtype=torch.int64, device=DEV)

    def call(self, out=None, lse=None, ws=None):
        return self.ctx.prepare_attend_shared(self.kv, self.q, self.pos_d, self.seq_d, self.order_d, self.head_d, self.shared_d,
                                              self.out if out is None else out, self.ws if ws is None else ws,
                                              sink=self.sink, lse=self.lse if lse is None else lse)

    def run(self, flags=0):
        self.call().run()
        got, _ = self.ctx.check()
        assert got == flags, f"flags {got:#x}"
        return self

    def views(self):
        """Each query's table row as the operator reads it."""
        views = [None] * len(self.seq)
        for k, i in enumerate(self.order):
            b = self.seq[i] if 0 <= i < len(self.seq) else -1
            if not 0 <= b < len(self.table_rows):
                continue
            h = self.head[k]
            first = self.seq[self.order[h]]
            cols = max(0, self.shared[h]) // self.page if 0 <= first < len(self.table_rows) else 0
            views[i] = list(self.table_rows[first][:cols]) + list(self.table_rows[b][cols:])
        return views

    def check(self, only=None, values=None):
        v = page_values(self.codes, self.scales, self.fmt) if values is None else values
        views = self.views()
        who = [i for i in (range(len(self.seq)) if only is None else only) if views[i] is not None]
        check_attend(self.out[who], self.lse[who], v, [views[i] for i in who], self.page, self.q[who], [self.pos[i] for i in who],
                     list(range(len(who))), None, 0, 0, self.sink, self.ctx.cfg)
        return self


# ---------------------------------------------------------------- sizes

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_two_queries_of_one_prompt(fmt):
    Case([(8, [150, 190])], fmt=fmt, page=16).run().check()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513])
def test_one_query_of_its_own(n):
    Case([(0, [n])], page=16, seed=n).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 256])
def test_page_sizes(fmt, page):
    whole = max(1, 320 // page)
    Case([(whole, [whole * page + 1, whole * page + 70, whole * page + 5]), (0, [33, 300])], fmt=fmt, page=page, seed=page).run().check()


@pytest.mark.parametrize("shared", [0, 1, 3, 4, 5, 16, 17])
@pytest.mark.parametrize("tails", [(1, 1), (1, 200), (64, 65), (63, 129, 10)])
def test_common_rows_and_tails(shared, tails):
    Case([(shared, [16 * shared + t for t in tails])], page=16, seed=shared + len(tails)).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("sizes", [(1, 2, 5, 3), (7,), (1, 1, 1), (2, 4)])
def test_groups_of_unlike_sizes(fmt, sizes):
    rng = random.Random(len(sizes))
    Case([(rng.randint(1, 9), [16 * 9 + rng.randint(1, 200) for _ in range(k)]) for k in sizes], fmt=fmt, page=16, seed=3,
         shuffle=True).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_long_prompt_is_split_over_many_pairs(fmt):
    Case([(160, [160 * 64 + 40, 160 * 64 + 700, 160 * 64 + 3])], fmt=fmt, page=64, seed=5).run().check()


def test_more_tiles_than_two_a_pair():
    Case([(40, [40 * 64 + 1 + 7 * i for i in range(30)]), (8, [8 * 64 + 5 * i + 1 for i in range(9)])], page=64,
         seed=6).run().check(only=[0, 1, 7, 14, 29, 30, 33, 38])


@pytest.mark.parametrize("per", [2, 3])
def test_several_queries_of_a_sequence(per):
    Case([(6, [16 * 6 + 20, 16 * 6 + 60, 16 * 6 + 3]), (0, [100])], page=16, per=per, seed=7).run().check()


def test_prompt_chunk_of_one_sequence():
    n = 333
    Case([(0, [n])], page=16, queries=[(0, t) for t in range(n - 130, n)], seed=8).run().check(only=list(range(0, 130, 9)) + [1, 129])


def test_prompt_chunk_from_an_empty_cache():
    Case([(0, [37])], page=8, queries=[(0, t) for t in range(37)], seed=9).run().check()


# ---------------------------------------------------------------- plans

def test_places_in_any_order():
    c = Case([(4, [100, 90, 80, 70, 77])], page=16, seed=10)
    c.order, c.head, c.shared = [4, 0, 3, 1, 2], [0, 0, 0, 3, 3], [64, 0, 0, 48, 0]
    c.plan()
    c.run().check()


def test_common_rows_come_from_the_groups_first_query():
    # rows of two unrelated sequences: below the common length only the first one's are read
    c = Case([(0, [200, 210])], page=16, seed=11)
    c.order, c.head, c.shared = [1, 0], [0, 0], [96, 0]
    c.plan()
    c.run().check()


@pytest.mark.parametrize("shared", [7, 16, 40, 1000, 1 << 40, -3])
def test_lengths_that_are_cut(shared):
    # not whole pages, past the queries' positions, past the table, below zero
    c = Case([(3, [60, 70, 90])], page=16, seed=12)
    c.shared[0] = shared
    c.plan()
    c.call().run()
    c.shared[0] = min(max(shared, 0), 16 * len(c.table_rows[0]))
    flags, _ = c.ctx.check()
    c.check()


def test_positions_below_the_common_length():
    c = Case([(10, [160, 170, 180])], page=16, queries=[(0, 159), (1, 20), (2, 101)], seed=13)
    c.run().check()


def test_empty_places_and_unlisted_queries_keep_their_outputs():
    c = Case([(2, [40, 50, 60, 70])], page=16, seed=14)
    c.order = [0, -1, 2, -1]
    c.head, c.shared = [0, 0, 2, 2], [32, 0, 32, 0]
    c.plan()
    c.run().check(only=[0, 2])
    assert (c.out[[1, 3]] == 77).all() and (c.lse[[1, 3]] == 77).all()


def test_padding_queries_stay_as_they_were():
    c = Case([(3, [50, 60, 70])], page=16, queries=[(0, 49), (-1, 5), (1, 59), (-1, -1), (2, 69)], seed=15)
    c.run().check(only=[0, 2, 4])
    assert (c.out[[1, 3]] == 77).all() and (c.lse[[1, 3]] == 77).all()
    # as a member of a group, and as its first place
    c.order, c.head, c.shared = [1, 0, 2, 3, 4], [0, 0, 0, 0, 0], [48, 0, 0, 0, 0]
    c.plan()
    c.run().check(only=[0, 2, 4])


def test_bad_queries_are_recorded_and_zero():
    c = Case([(1, [30, 40])], page=16, queries=[(0, 29), (2, 5), (-7, 3), (1, -2), (1, 39)], seed=16)
    c.run(flags=c.b.FLAG_BAD_QUERY).check(only=[0, 4])
    for i in (1, 2, 3):
        assert (c.out[i] == 0).all()
        assert torch.equal(c.lse[i], c.sink)


def test_queries_that_see_nothing():
    c = Case([(1, [30, 40])], page=16, queries=[(0, -1), (1, 39), (0, 29), (1, -1), (0, -1)], seed=17)
    c.run().check()
    for i in (0, 3, 4):
        assert (c.out[i] == 0).all() and torch.equal(c.lse[i], c.sink)


def test_bad_places_are_recorded():
    c = Case([(2, [40, 50, 60, 70])], page=16, seed=18)
    c.order, c.head, c.shared = [0, 99, 2, -5], [0, 0, 2, 2], [32, 0, 32, 0]
    c.plan()
    c.run(flags=c.b.FLAG_BAD_QUERY).check(only=[0, 2])
    # heads behind their place, negative, or of another group: every place is a group, or left out
    c.order, c.head, c.shared = [0, 1, 2, 3], [3, -4, 0, 2], [32, 0, 32, 0]
    c.plan()
    c.out.fill_(77)
    c.call().run()
    flags, _ = c.ctx.check()
    assert flags & ~c.b.FLAG_BAD_QUERY == 0
    assert torch.isfinite(c.out).all()


@pytest.mark.parametrize("sink", [None, -math.inf, 30.0])
def test_sinks(sink):
    s = None if sink is None else torch.full((HEADS,), sink, device=DEV)
    Case([(3, [60, 90, 49])], sink=s, seed=19).run().check()


def test_context_without_rope():
    Case([(3, [60, 90, 49])], rope=False, seed=20).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_strided_pages_and_tables(fmt):
    Case([(3, [60, 90, 49]), (0, [120])], fmt=fmt, layers=3, extra_cols=5, seed=21).run().check()


# ---------------------------------------------------------------- values

@pytest.mark.parametrize("page", [4, 16])
def test_large_scores_move_the_reference(page):
    c = Case([(512 // page, [530, 700, 512 + 140])], page=page, q_scale=3.0, seed=22)
    for k, at in enumerate((3, 300, 511, 560, 690)):
        g = c.table_rows[1][at // page]
        c.codes[g, at % page] *= 4 * (k + 1)
    c.run().check()


def test_first_rows_that_score_far_below_the_later_ones():
    c = Case([(32, [520, 600])], page=16, q_scale=8.0, seed=23)
    q = c.q[0].float().mean(0)
    for at in range(512):
        c.codes[c.table_rows[0][at // 16], at % 16] = (q * (-4.0 if at < 256 else 4.0)).to(torch.bfloat16)
    c.run().check()


@pytest.mark.parametrize("power", [80, -80])
def test_rows_far_from_unit_size(power):
    c = Case([(8, [150, 190])], page=16, seed=24, sink=None)
    c.codes.mul_(2.0 ** power)
    c.q.mul_(2.0 ** -power)
    c.run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [4, 16, 64])
def test_nan_in_rows_that_are_not_seen(fmt, page):
    # behind every length, and in a page that no sequence has
    c = Case([(3, [3 * page + 2, 3 * page + page // 2 + 1, 5 * page]), (0, [page + 1])], fmt=fmt, page=page, seed=25)
    clean = page_values(c.codes, c.scales, c.fmt)
    used = torch.zeros(c.codes.shape[:2], dtype=torch.bool)
    for row, n in zip(c.table_rows, c.lens):
        for p in range(n):
            used[row[p // page], p % page] = True
    hole = (~used).to(DEV)
    if fmt == "bf16":
        c.codes[hole] = math.nan
    elif fmt == "fp8":
        c.codes[hole] = 0x7F
    else:
        c.scales[hole] = 0x7F
    c.run().check(values=clean)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", [0, 1])
def test_a_row_of_one_query_leaves_the_other_alone(value, which):
    # tails in the same tile: the other query's weights there are zeros, which times a NaN are none
    c = Case([(4, [64 + 30, 64 + 100])], page=16, seed=26)
    at = c.lens[which] - 5
    clean = page_values(c.codes, c.scales, c.fmt)
    c.codes[c.table_rows[which][at // 16], at % 16] = value
    c.run().check(only=[1 - which], values=clean)
    assert not torch.isfinite(c.out[which]).all()


@pytest.mark.parametrize("which", [0, 1])
def test_a_query_of_nans_leaves_its_neighbours_alone(which):
    c = Case([(20, [330, 350, 321])], page=16, seed=27)
    c.q[which] = math.nan
    c.run().check(only=[i for i in range(3) if i != which])
    assert torch.isnan(c.out[which]).all() and torch.isnan(c.lse[which]).all()


def test_a_position_that_only_the_later_query_sees():
    # two queries of a sequence, the row between them not finite
    c = Case([(0, [100])], page=16, queries=[(0, 98), (0, 99)], seed=28)
    clean = page_values(c.codes, c.scales, c.fmt)
    c.codes[c.table_rows[0][99 // 16], 99 % 16] = math.nan
    c.run().check(only=[0], values=clean)


def test_missing_pages_are_left_out_and_recorded():
    c = Case([(6, [16 * 6 + 40, 16 * 6 + 90, 16 * 6 + 20])], page=16, seed=29)
    for row, col in ((0, 2), (1, 2), (1, 7), (2, 6)):
        c.table_rows[row][col] = -1 if col != 7 else 10 ** 6
        c.table[row, col] = c.table_rows[row][col]
    c.run(flags=c.b.FLAG_BAD_PAGE).check()


def test_every_row_missing():
    c = Case([(2, [40, 50])], page=16, seed=30)
    c.table.fill_(-1)
    c.run(flags=c.b.FLAG_BAD_PAGE)
    assert (c.out == 0).all() and torch.equal(c.lse, c.sink.expand_as(c.lse))


def test_positions_past_the_table():
    c = Case([(2, [48, 48])], page=16, queries=[(0, 100), (1, 1 << 40)], seed=31)
    c.run(flags=c.b.FLAG_BAD_PAGE)
    c.pos = [47, 47]
    v = page_values(c.codes, c.scales, c.fmt)
    # the rows that are there, rotated at the far positions: the output's plain channels and lse against a context's own bound
    from paged_common import attend_one
    for i, t in enumerate((100, 1 << 40)):
        if i == 1:
            continue
        o, l, bo, bl = attend_one(v, c.views()[i], 16, c.q[i], t, 0, 0, 0, c.sink, c.ctx.cfg)
        assert ((c.out[i].double().cpu() - o).abs() <= bo).all()
        assert ((c.lse[i].double().cpu() - l).abs() <= bl).all()


def test_page_offsets_past_32_bits():
    # pages 5 GB apart from the first: byte offsets past 2^32
    page, n_pages = 64, 70000
    c = Case([(2, [150, 170])], page=page, seed=32, spare=8)
    big = torch.zeros((n_pages, page, DIM), dtype=torch.bfloat16, device=DEV)
    far = [n_pages - 1 - i for i in range(c.codes.shape[0])]
    big[far] = c.codes
    c.table_rows = [[far[g] if g >= 0 else -1 for g in r] for r in c.table_rows]
    c.table = torch.tensor(c.table_rows, dtype=torch.int32, device=DEV)
    small = page_values(c.codes, c.scales, c.fmt)
    c.codes = big
    c.kv = c.ctx.paged_kv(big, c.table)
    c.call().run()
    assert c.ctx.check()[0] == 0
    back = {f: i for i, f in enumerate(far)}
    c.table_rows = [[back[g] if g >= 0 else -1 for g in r] for r in c.table_rows]
    c.check(values=small)


# ---------------------------------------------------------------- calls

@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_repeats_bit_for_bit_and_on_another_stream(fmt):
    c = Case([(30, [30 * 64 + 50 * i + 1 for i in range(5)]), (3, [300, 500])], fmt=fmt, page=64, seed=33).run()
    out, lse = c.out.clone(), c.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            c.out.fill_(77)
            c.lse.fill_(77)
            c.call().run()
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


def test_two_calls_at_once_with_a_workspace_each():
    a = Case([(20, [1300, 1400, 1290])], page=64, seed=34)
    b = Case([(9, [600, 620]), (0, [100])], page=64, seed=35)
    other = a.b.Context()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    b.ctx, b.kv = other, other.paged_kv(b.codes, b.table)
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(s):
                c.call().run()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_captured_graph_follows_the_state():
    c = Case([(8, [16 * 8 + 30, 16 * 8 + 90, 16 * 8 + 3])], page=16, seed=36)
    c.run()
    call = c.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
        call.run()  # one workspace, one after another
    c.pos = [16 * 8 + 3, 16 * 8 + 60, 5]
    c.pos_d.copy_(torch.tensor(c.pos))
    c.shared[0] = 16 * 5
    c.shared_d.copy_(torch.tensor(c.shared))
    c.out.fill_(77)
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_no_queries_enqueue_nothing():
    c = Case([(1, [20])])
    none = c.ctx.prepare_attend_shared(c.kv, c.q[:0], c.pos_d[:0], c.seq_d[:0], c.order_d[:0], c.head_d[:0], c.shared_d[:0],
                                       c.out[:0], c.ws)
    none.run()
    assert c.ctx.last_launch_count == 0


def test_refusals():
    c = Case([(1, [20, 30])])
    def call(**kw):
        a = dict(q=c.q, q_pos=c.pos_d, seq_of_q=c.seq_d, order=c.order_d, head=c.head_d, shared=c.shared_d, out=c.out,
                 workspace=c.ws)
        a.update(kw)
        c.ctx.attend_shared(c.kv, a["q"], a["q_pos"], a["seq_of_q"], a["order"], a["head"], a["shared"], a["out"], a["workspace"])
    for kw in (dict(q=c.q.float()), dict(q_pos=c.pos_d.int()), dict(order=c.order_d.long()), dict(shared=c.shared_d.int()),
               dict(head=c.head_d.cpu()), dict(order=None), dict(head=None), dict(shared=None), dict(out=None)):
        with pytest.raises((TypeError, ValueError, AttributeError, c.b.Csa2Error)):
            call(**kw)
    for kw in (dict(order=c.order_d[:1]), dict(shared=c.shared_d[:1]), dict(out=c.out[:1])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(c.b.Csa2Error, match="workspace"):
        call(workspace=c.ws[:1000])
    with pytest.raises(c.b.Csa2Error, match="aligned"):
        call(workspace=torch.empty(c.ws.numel() + 512, dtype=torch.uint8, device=DEV)[1:])
    with pytest.raises(c.b.Csa2Error, match="overlaps"):
        call(out=c.q)
    both = torch.empty((3, HEADS, DIM), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(c.b.Csa2Error, match="overlaps"):
        call(q=both[:2], out=both[1:])
    with pytest.raises(c.b.Csa2Error):
        c.kv = c.ctx.paged_kv(c.codes)  # a cache without a table
        call()
    with pytest.raises(ValueError):
        c.kv = context(kv_format="fp8").paged_kv(torch.zeros((2, 16, 512), dtype=torch.uint8, device=DEV), c.table,
                                                 torch.zeros((2, 16, 16), dtype=torch.uint8, device=DEV))
        call()


def test_lse_may_be_left_out():
    c = Case([(2, [40, 50])], seed=37)
    c.ctx.attend_shared(c.kv, c.q, c.pos_d, c.seq_d, c.order_d, c.head_d, c.shared_d, c.out, c.ws, sink=c.sink)
    out = c.out.clone()
    c.run().check()
    assert torch.equal(out, c.out)


def test_many_queries():
    n = 2500
    rng = random.Random(38)
    c = Case([(0, [40 + rng.randint(0, 100)]) for _ in range(50)], page=16, seed=38,
             queries=[(i % 50, rng.randint(0, 39)) for i in range(n)])
    c.run().check(only=rng.sample(range(n), 40))


@pytest.mark.parametrize("n", [75, 76, 77, 95, 96, 97, 200])
def test_numbers_of_queries_around_the_plans(n):
    # the plan is made by every pair of CTAs or by a launch of its own, and joins are kept by unit or by run
    rng = random.Random(n)
    groups, left = [], n
    while left:
        k = min(left, rng.choice([1, 1, 2, 3, 8, 20]))
        whole = rng.choice([0, 3, 12, 60])
        groups.append((whole, [16 * whole + rng.randint(1, 300) for _ in range(k)]))
        left -= k
    c = Case(groups, page=16, seed=n, shuffle=True).run()
    c.check(only=rng.sample(range(n), 30))


@pytest.mark.parametrize("n", [100, 1100, 2300])
def test_one_long_query_among_many_short_ones(n):
    # units that other runs begin and end in, and one over many pairs of CTAs
    lens = [9000] + [1 + i % 40 for i in range(19)]
    queries = [(1 + i % 19, (i % 19) % 40) for i in range(n - 1)]
    queries.insert(n // 2, (0, 8999))
    c = Case([(0, [m]) for m in lens], page=16, seed=n, queries=queries)
    c.run().check(only=[0, 1, n // 2 - 1, n // 2, n // 2 + 1, n - 1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_groups_ends_in_every_place_of_a_page(fmt):
    # tails that end 1 .. 64 rows into their last group, in one call
    Case([(4, [256 + 1 + i for i in range(0, 64, 3)])], fmt=fmt, page=64, seed=40).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [8, 32, 128, 4096])
def test_empty_and_single_row_queries_beside_long_ones(fmt, page):
    Case([(0, [1, 2 * page, 300])], fmt=fmt, page=page, queries=[(0, -1), (2, 299), (0, 0), (1, 0), (1, 2 * page - 1), (2, 64)],
         seed=41).run().check()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_nan_codes_are_not_numbers(fmt):
    # a visible row of NaN codes or scales reaches the queries that see it, and no others
    c = Case([(3, [64 * 3 + 20, 64 * 3 + 50, 64 * 3 + 5])], fmt=fmt, page=64, seed=42)
    clean = page_values(c.codes, c.scales, c.fmt)
    at = c.lens[1] - 2
    (c.codes if fmt == "fp8" else c.scales)[c.table_rows[1][at // 64], at % 64] = 0x7F
    c.run().check(only=[0, 2], values=clean)
    assert torch.isnan(c.out[1]).any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_the_first_call_of_a_host_thread(fmt):
    import threading
    c = Case([(3, [100, 200])], fmt=fmt, page=16, seed=43).run()
    want, call, bad = c.out.clone(), c.call(), []
    c.out.zero_()
    torch.cuda.synchronize()

    def work():
        try:
            call.run()
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_agrees_with_attend_paged_on_its_own_groups(fmt):
    """Groups found by csa2_query_groups, the result against csa2_attend_paged's
    on the same queries: both within their bounds of the exact result."""
    c = Case([(7, [16 * 7 + 30, 16 * 7 + 9, 16 * 7 + 77]), (5, [16 * 5 + 3, 16 * 5 + 40]), (0, [90])], fmt=fmt, page=16, per=2, seed=44)
    n = len(c.seq)
    order, head = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
    shared = torch.empty(n, dtype=torch.int64, device=DEV)
    c.ctx.query_groups(c.table, 16, c.codes.shape[0], c.pos_d, c.seq_d, 40, order, head, shared)
    c.order, c.head, c.shared = order.tolist(), head.tolist(), shared.tolist()
    assert c.shared[0] == 16 * 7 and c.shared[6] == 16 * 5
    c.plan()
    c.run().check()
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    ws = c.b.workspace(c.ctx.attend_paged_workspace_size(n), DEV)
    c.ctx.attend_paged(c.kv, c.q, c.pos_d, c.seq_d, out, ws, sink=c.sink, lse=lse)
    # twice attend_one's lse bound: 40 U32 of a score's sum of sizes (below 64 here), 2^-21 and 8 U32 of its own size
    assert ((lse - c.lse).abs() <= 2 * (40 * U32 * 64 + 2.0 ** -16 * 4 + 2.0 ** -21 + 8 * U32 * (1 + lse.abs()))).all()


def test_misaligned_buffers_are_refused():
    c = Case([(1, [20, 30])])
    lib, p = c.b.load_library(), lambda t: t.data_ptr()
    import ctypes as C
    good = [p(c.q), p(c.pos_d), p(c.seq_d), p(c.order_d), p(c.head_d), p(c.shared_d), p(c.sink), p(c.out), p(c.lse)]
    for i, step in enumerate((8, 4, 2, 2, 2, 4, 2, 8, 2)):
        a = list(good)
        a[i] += step
        st = lib.csa2_attend_shared(c.ctx.h, None, C.byref(c.kv.args), 2, *a, p(c.ws), c.ws.numel())
        assert st == 1, i
        assert c.ctx.last_launch_count == 0
