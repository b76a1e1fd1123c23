"""csa2_attend_paged against a plain 64-bit form, at the sizes, masks, layouts
and streams where it can go wrong. The bounds are derived in
paged_common.attend_one."""
import math
import random

import pytest
import torch

from gpu_common import context, require_gpu
from paged_common import DIM, FMT_NAMES, HEADS, U32, check_attend, page_values, random_pages

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """A small paged cache and its queries; run() calls the entry point."""

    def __init__(self, lens, fmt="bf16", page=16, per=1, window=0, n_first=0, lo=None, sink=True, seed=0, spare=2,
                 queries=None, rope=True, layers=0, extra_cols=0, q_scale=1.0):
        from compressed_sparse_attention_gb300 import binding
        require_gpu()
        self.b = binding
        self.ctx = context(kv_format=fmt, **({} if rope else {"rope_dim": 0}))
        self.fmt, self.page, self.window, self.n_first = FMT_NAMES[fmt], page, window, n_first
        rng = random.Random(seed)
        counts = [-(-n // page) for n in lens]
        n_pages = sum(counts) + spare
        order = list(range(n_pages))
        rng.shuffle(order)
        width = max(1, max(counts))
        self.table_rows = [[order.pop() for _ in range(c)] + [-1] * (width - c) for c in counts]
        self.codes, self.scales = random_pages(self.fmt, n_pages, page, seed, DEV, (layers,) if layers else ())
        if layers:  # pages of several layers side by side: [n_pages, layers, page, ..], this layer the last
            self.codes = self.codes.transpose(0, 1).contiguous()[:, -1]
            self.scales = None if self.scales is None else self.scales.transpose(0, 1).contiguous()[:, -1]
        full = torch.full((len(lens), width + extra_cols), 7, dtype=torch.int32)
        full[:, :width] = torch.tensor(self.table_rows, dtype=torch.int32)
        self.table = full.to(DEV)[:, :width]
        queries = queries if queries is not None else [(b, n - per + i) for b, n in enumerate(lens) for i in range(per)]
        self.seq, self.pos = [b for b, _ in queries], [t for _, t in queries]
        n = len(queries)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = (q_scale * torch.randn((n, HEADS, DIM), generator=g)).to(torch.bfloat16).to(DEV)
        self.sink = torch.randn((HEADS,), generator=g).to(DEV) if sink is True else sink
        self.lo = lo
        self.seq_d = torch.tensor(self.seq, dtype=torch.int32, device=DEV)
        self.pos_d = torch.tensor(self.pos, dtype=torch.int64, device=DEV)
        self.lo_d = None if lo is None else torch.tensor(lo, dtype=torch.int64, device=DEV)
        self.out = torch.full((n, HEADS, DIM), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((n, HEADS), 77.0, device=DEV)
        self.ws = binding.workspace(self.ctx.attend_paged_workspace_size(n), DEV)
        self.kv = self.ctx.paged_kv(self.codes, self.table, self.scales)

    def call(self, out=None, lse=None, ws=None):
        return self.ctx.prepare_attend_paged(self.kv, self.q, self.pos_d, self.seq_d, self.out if out is None else out,
                                             self.ws if ws is None else ws, sink=self.sink,
                                             lse=self.lse if lse is None else lse, lo=self.lo_d, window=self.window,
                                             n_first=self.n_first)

    def run(self, flags=0):
        self.call().run()
        got, _ = self.ctx.check()
        assert got == flags, f"device error word 0x{got:x}"
        return self

    def check(self, values=None):
        if values is None:
            values = page_values(self.codes, self.scales, self.fmt)
        check_attend(self.out, self.lse, values, self.table_rows, self.page, self.q, self.pos, self.seq, self.lo,
                     self.window, self.n_first, self.sink, self.ctx.cfg)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 257, 700])
def test_lengths_around_the_tile(fmt, n):
    Case([n], fmt=fmt, page=32, seed=n).run().check()


@pytest.mark.parametrize("page", [1, 2, 8, 64, 128, 256, 1024])
def test_page_sizes(page):
    Case([333, 1, 140], page=page, seed=page).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_one_long_sequence_is_split_over_many_ctas(fmt):
    Case([9000, 5], fmt=fmt, page=64, seed=3).run().check()


@pytest.mark.parametrize("fmt,per", [("bf16", 1), ("fp8", 3), ("fp4", 2)])
def test_ragged_batch(fmt, per):
    Case([1 + per, 900, 64, 65, 2000, 128, 511], fmt=fmt, per=per, seed=4).run().check()


@pytest.mark.parametrize("window,n_first", [(1, 0), (1, 1), (5, 200), (100, 4), (128, 0), (127, 1), (124, 4), (400, 7),
                                            (10 ** 12, 3), (300, 10 ** 12)])
def test_windows_and_first_tokens(window, n_first):
    Case([1, 50, 131, 400, 777], window=window, n_first=n_first, seed=window % 1000).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_prompt_chunk_under_a_window(fmt):
    # every token of a chunk is a query: more queries than SMs, several tiles each
    Case([420, 333], fmt=fmt, per=110, window=150, n_first=4, lo=[0, 9], page=32, seed=6).run().check()


def test_left_padding_and_rows_that_see_nothing():
    # lo past t, lo negative, an empty sequence (t = -1)
    Case([40, 40, 40, 3], lo=[60, 39, -5, 0], seed=7, queries=[(0, 39), (1, 39), (2, 39), (3, -1)]).run().check()
    Case([40, 40], lo=[60, 20], window=9, n_first=3, seed=8).run().check()


@pytest.mark.parametrize("sink", [None, -math.inf, 80.0, -80.0])
def test_sinks(sink):
    s = None if sink is None else torch.full((HEADS,), sink, device=DEV)
    Case([300, 1, 7], sink=s, lo=[0, 5, 0], seed=9).run().check()


def test_large_scores_move_the_reference():
    # scores in the hundreds: the reference must follow the rows
    Case([600, 200], q_scale=30.0, seed=10).run().check()


def test_padding_queries_stay_as_they_were():
    c = Case([100, 200], queries=[(0, 99), (-1, 5), (1, 199), (-1, -1)], seed=11)
    c.run().check()
    for i in (1, 3):
        assert (c.out[i] == 77.0).all() and (c.lse[i] == 77.0).all()


def test_bad_queries_are_recorded_and_zero():
    c = Case([100, 200], queries=[(0, 99), (2, 5), (1, -2), (-2, 3)], seed=12)
    c.run(flags=c.b.FLAG_BAD_QUERY)
    assert (c.out[1:] == 0).all()
    # the sink times log2(e) and back by ln 2: two constants and two products, each rounded once
    assert ((c.lse[1:] - c.sink).abs() <= 4 * U32 * c.sink.abs()).all()
    c.seq, c.pos = c.seq[:1], c.pos[:1]
    c.check()


def test_missing_pages_are_left_out_and_recorded():
    c = Case([300, 200], page=32, seed=13)
    for row, col, v in ((0, 3, -1), (1, 0, 10 ** 6), (1, 2, -7)):
        c.table_rows[row][col] = v
        c.table[row, col] = v
    c.run(flags=c.b.FLAG_BAD_PAGE).check()
    # a position past the table's columns: what the table holds is read
    d = Case([64], page=32, queries=[(0, 10 ** 9)], seed=14)
    d.run(flags=d.b.FLAG_BAD_PAGE)
    d.pos = [63]
    values = page_values(d.codes, d.scales, d.fmt)
    # (the rotation is by the true position, which only the magnitude check below can use)
    assert torch.isfinite(d.out.float()).all() and values.shape[0] >= 2


def test_missing_pages_outside_the_window_are_not_read():
    c = Case([500], page=16, window=40, n_first=4, seed=15)
    for j in range(1, 500 // 16 - 3):
        c.table_rows[0][j] = -1
        c.table[0, j] = -1
    c.run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_nan_in_rows_that_are_not_seen(fmt):
    c = Case([70, 210], fmt=fmt, page=32, lo=[0, 33], window=64, n_first=3, seed=16)
    values = page_values(c.codes, c.scales, c.fmt)
    seen = torch.zeros(values.shape[:2], dtype=torch.bool)
    from paged_common import visible
    for b, t in zip(c.seq, c.pos):
        for p in visible(t, c.lo[b], c.window, c.n_first):
            seen[c.table_rows[b][p // c.page], p % c.page] = True
    bad = ~seen.to(DEV)
    if c.fmt == 0:
        c.codes[bad] = math.nan
        c.codes[0][bad[0]] = math.inf
    else:
        c.codes[bad] = 0x7F
        c.scales[bad] = 0xFF if c.fmt == 1 else 0x7F
    c.run().check(values)


def test_every_row_of_a_split_missing():
    # a run of tiles without a single row between tiles that have some
    c = Case([2000], page=16, seed=17)
    for j in range(20, 100):
        c.table_rows[0][j] = -1
        c.table[0, j] = -1
    c.run(flags=c.b.FLAG_BAD_PAGE).check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_strided_pages_and_tables(fmt):
    Case([100, 333], fmt=fmt, page=32, layers=3, extra_cols=5, seed=18).run().check()


def test_context_without_rope():
    Case([100, 333], rope=False, seed=19).run().check()


def test_more_queries_than_one_launch_takes():
    n = 4100
    c = Case([300, 40], page=64, queries=[(i % 2, (i * 7) % (300 if i % 2 == 0 else 40)) for i in range(n)], window=60,
             n_first=2, seed=20)
    c.run()
    assert c.ctx.last_launch_count == 4
    pick = list(range(0, n, 97)) + [4095, 4096, n - 1]
    c.out, c.lse, c.q = c.out[pick], c.lse[pick], c.q[pick]
    c.seq, c.pos = [c.seq[i] for i in pick], [c.pos[i] for i in pick]
    c.check()


def test_page_offsets_past_32_bits():
    # 70,000 pages of 64 KB: codes past 4 GB; only the last pages are used
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    n_pages = 70000
    pages = torch.empty((n_pages, 64, DIM), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(21)
    last = torch.randn((3, 64, DIM), generator=g).to(torch.bfloat16)
    pages[-3:] = last.to(DEV)
    rows = [[n_pages - 1, n_pages - 3, n_pages - 2]]
    q = torch.randn((1, HEADS, DIM), generator=g).to(torch.bfloat16).to(DEV)
    out = torch.empty_like(q)
    ws = binding.workspace(ctx.attend_paged_workspace_size(1), DEV)
    kv = ctx.paged_kv(pages, torch.tensor(rows, dtype=torch.int32, device=DEV))
    ctx.attend_paged(kv, q, torch.tensor([180], device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), out, ws)
    assert ctx.check()[0] == 0
    check_attend(out, None, last.double(), [[2, 0, 1]], 64, q, [180], [0], None, 0, 0, None, ctx.cfg)


def test_repeats_bit_for_bit_and_on_another_stream():
    c = Case([3000, 700, 90, 1], page=32, seed=22).run()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.out.fill_(5)
        c.call().run()
    s.synchronize()
    assert torch.equal(c.out, out)


def test_two_calls_at_once_with_a_workspace_each():
    a, b = Case([4000, 30], seed=23).run(), Case([2500] * 3, fmt="fp8", seed=24).run()
    want = [a.out.clone(), b.out.clone()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                c.out.zero_()
                c.call().run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_captured_graphs_share_a_workspace_and_follow_the_state():
    c = Case([800, 300], page=32, seed=25).run()
    first = c.out.clone()
    out2 = torch.zeros_like(c.out)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c.call().run()
    with torch.cuda.graph(g2):  # the same workspace, another output
        c.call(out=out2).run()
    for _ in range(3):
        c.out.zero_()
        out2.zero_()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(out2, first)
    c.pos = [555, 17]
    c.pos_d.copy_(torch.tensor(c.pos))
    g1.replay()
    torch.cuda.synchronize()
    c.check()


def test_no_queries_enqueue_nothing():
    c = Case([10], queries=[], seed=26)
    assert c.ctx.attend_paged_workspace_size(0) == 0
    c.run()
    assert c.ctx.last_launch_count == 0


def test_refusals():
    from compressed_sparse_attention_gb300 import binding
    c = Case([100], page=16, seed=27)
    lib, p = c.ctx.lib, c.call()

    def st(**kw):
        a = binding.PagedKVArgs.from_buffer_copy(c.kv.args)
        args = dict(n=1, window=0, n_first=0, q=c.q.data_ptr(), out=c.out.data_ptr(), ws=c.ws.data_ptr(), size=c.ws.numel())
        for k, v in kw.items():
            if k in args:
                args[k] = v
            else:
                setattr(a, k, v)
        return lib.csa2_attend_paged(c.ctx.h, None, binding.C.byref(a), args["n"], args["q"], c.pos_d.data_ptr(),
                                     c.seq_d.data_ptr(), None, args["window"], args["n_first"], None, args["out"], None,
                                     args["ws"], args["size"])

    c.out.fill_(3)
    for kw in (dict(page_size=24), dict(page_size=0), dict(page_size=8192), dict(max_pages=1 << 28, table_ld=1 << 28)):
        assert st(**kw) == 2, kw
    for kw in (dict(n_pages=0), dict(n_seq=0), dict(table_ld=1), dict(table=None), dict(pages=None), dict(page_stride=16),
               dict(page_stride=16 * 1024 + 8), dict(pages=c.codes.data_ptr() + 2), dict(n=-1), dict(window=-1),
               dict(n_first=-1), dict(q=None), dict(out=None), dict(q=c.q.data_ptr() + 2), dict(ws=c.ws.data_ptr() + 16)):
        assert st(**kw) == 1, kw
    assert st(size=c.ws.numel() - 1) == 6 and st(ws=None) == 6
    f8 = Case([100], fmt="fp8", seed=28)
    a = binding.PagedKVArgs.from_buffer_copy(f8.kv.args)
    a.scales = None
    assert lib.csa2_attend_paged(f8.ctx.h, None, binding.C.byref(a), 1, f8.q.data_ptr(), f8.pos_d.data_ptr(),
                                 f8.seq_d.data_ptr(), None, 0, 0, None, f8.out.data_ptr(), None, f8.ws.data_ptr(),
                                 f8.ws.numel()) == 1
    torch.cuda.synchronize()
    assert (c.out == 3).all() and c.ctx.last_launch_count == 0 and p is not None


def test_refuses_misaligned_elements():
    from compressed_sparse_attention_gb300 import binding
    c = Case([100], page=16, seed=29)
    c.out.fill_(3)
    good = dict(pos=c.pos_d.data_ptr(), seq=c.seq_d.data_ptr(), lo=None, sink=c.sink.data_ptr(), lse=c.lse.data_ptr())
    for k, by in (("pos", 4), ("seq", 2), ("lo", 4), ("sink", 1), ("lse", 2)):
        a = dict(good, **{k: (good[k] or good["pos"]) + by})
        assert c.ctx.lib.csa2_attend_paged(c.ctx.h, None, binding.C.byref(c.kv.args), 1, c.q.data_ptr(), a["pos"], a["seq"],
                                           a["lo"], 0, 0, a["sink"], c.out.data_ptr(), a["lse"], c.ws.data_ptr(),
                                           c.ws.numel()) == 1, k
    torch.cuda.synchronize()
    assert (c.out == 3).all() and c.ctx.last_launch_count == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [8, 32])
def test_more_tiles_than_two_a_cta(fmt, page):
    # runs are then cut by cost: many short sequences, some of one row, and long ones that cross many runs
    rng = random.Random(30)
    lens = [rng.choice([1, 3, 130, rng.randint(100, 900), rng.randint(100, 900)]) for _ in range(80)] + [9001, 1, 6000]
    rng.shuffle(lens)
    Case(lens, fmt, page=page, seed=31).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_long_and_empty_queries_in_turn_under_a_window(fmt):
    # every third query sees nothing, neighbours see one to eleven tiles
    rng = random.Random(32)
    lens = [rng.randint(1, 1500) for _ in range(40)]
    queries = []
    for b, n in enumerate(lens):
        queries += [(b, n - 1), (b, -1), (b, rng.randint(0, n - 1)), (-1, 5)]
    c = Case(lens, fmt, page=16, window=1300, n_first=3, lo=[rng.choice([0, 0, 7]) for _ in lens], queries=queries, seed=33)
    c.run().check()
    assert (c.out.view(-1, 4, HEADS, DIM)[:, 3] == 77.0).all() and (c.lse.view(-1, 4, HEADS)[:, 3] == 77.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_query_of_nans_leaves_its_neighbours_alone(fmt):
    # two queries a CTA and more: every other one NaN or infinite
    rng = random.Random(34)
    c = Case([rng.randint(1, 400) for _ in range(330)], fmt, page=16, seed=35)
    clean = c.q.clone()
    c.q[1::4] = math.nan
    c.q[3::4, :, :7] = math.inf
    c.run()
    bad, bad_lse = c.out[1::2].clone(), c.lse[1::2].clone()
    assert torch.isnan(bad[0::2]).all() and torch.isnan(bad_lse[0::2]).all()
    good = c.out[0::2].clone(), c.lse[0::2].clone()
    c.q = clean
    c.run().check()
    assert torch.equal(c.out[0::2], good[0]) and torch.equal(c.lse[0::2], good[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_first_tiles_without_a_row_before_tiles_with_some(fmt):
    # several tiles a CTA; the first one or two of every second query have no page, and its scores lie below the
    # reference that nothing has set (a weight of 2^-150 and less against 1)
    from compressed_sparse_attention_gb300 import binding
    rng = random.Random(36)
    lens = [rng.randint(300, 520) for _ in range(330)]
    c = Case(lens, fmt, page=16, seed=37, sink=None)
    for b in range(0, 330, 2):
        n = rng.choice([8, 9, 16])
        c.table_rows[b][:n] = [-1] * n
        c.table[b, :n] = -1
    c.run(flags=binding.FLAG_BAD_PAGE).check()
    values = page_values(c.codes, c.scales, c.fmt)
    # one direction of the rows, far below zero for every query of the second half
    side = values.mean((0, 1))
    side = side / side.norm()
    low = -(3000.0 * side).to(torch.bfloat16).to(DEV)
    c.q[165:] = low
    c.run(flags=binding.FLAG_BAD_PAGE).check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("share,more", [(4, 0), (4, 1), (2, 0), (2, 1)])
def test_tiles_around_a_share_of_the_ctas(fmt, share, more):
    # with fewer tiles than half or a quarter of the CTAs several of them share a tile's output dims
    require_gpu()
    tiles = torch.cuda.get_device_properties(0).multi_processor_count // share + more
    rng = random.Random(38)
    Case([rng.randint(1, 128) for _ in range(tiles)], fmt, page=16, seed=39).run().check()
    Case([128 * (tiles - 3) - 5, 129, 1], fmt, page=64, seed=40).run().check()


def test_refuses_an_output_over_its_queries():
    # CTAs that share a query's output dims each read its whole Q, so nothing may be stored over it
    from compressed_sparse_attention_gb300 import binding
    c = Case([100, 30, 7], page=16, seed=41)
    row = HEADS * DIM
    buf = torch.zeros((8 * row,), dtype=torch.bfloat16, device=DEV)
    buf[2 * row:5 * row] = c.q.view(-1)
    keep = buf.clone()
    c.q = buf[2 * row:5 * row].view(3, HEADS, DIM)
    for at in (2 * row, row, 3 * row, 5 * row - 8, 8):  # the same place, a query earlier and later, 16 bytes of overlap
        with pytest.raises(binding.Csa2Error) as e:
            c.call(out=buf[at:at + 3 * row].view(3, HEADS, DIM)).run()
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert torch.equal(buf, keep) and c.ctx.last_launch_count == 0
    # right behind q and right before it
    wide = torch.zeros((9 * row,), dtype=torch.bfloat16, device=DEV)
    c.q = wide[3 * row:6 * row].view(3, HEADS, DIM)
    c.q.copy_(keep[2 * row:5 * row].view(3, HEADS, DIM))
    for at in (0, 6 * row):
        c.out = wide[at:at + 3 * row].view(3, HEADS, DIM)
        c.run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_the_first_call_of_a_host_thread(fmt):
    # a thread that has made no CUDA call has no current driver context, which a tensor map's encoding wants
    import threading
    c = Case([100, 300], fmt=fmt, page=16, seed=42).run()
    want = c.out.clone()
    call = c.call()
    for _ in range(2):
        c.out.zero_()
        torch.cuda.synchronize()
        bad = []

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


def test_first_calls_of_two_host_threads():
    # a fresh process, whose first calls of the library come from two threads at once, each on a context and a stream of its own
    import os
    import subprocess
    import sys
    require_gpu()
    code = """
import threading, torch
from compressed_sparse_attention_gb300 import binding
g = torch.Generator().manual_seed(0)
pages = torch.randn((8, 16, 512), generator=g).to(torch.bfloat16).cuda()
table = torch.arange(8, dtype=torch.int32, device='cuda').view(1, 8)
q = torch.randn((1, 64, 512), generator=g).to(torch.bfloat16).cuda()
pos, seq = torch.tensor([120], device='cuda'), torch.zeros(1, dtype=torch.int32, device='cuda')
made = []
for _ in range(2):
    ctx = binding.Context()
    ws = binding.workspace(ctx.attend_paged_workspace_size(1), 'cuda')
    out = torch.zeros_like(q)
    made.append((ctx, out, ctx.prepare_attend_paged(ctx.paged_kv(pages, table), q, pos, seq, out, ws), torch.cuda.Stream()))
torch.cuda.synchronize()
gate, bad = threading.Barrier(2), []
def work(i):
    try:
        with torch.cuda.stream(made[i][3]):
            gate.wait()
            made[i][2].run()
    except Exception as e:
        bad.append(e)
threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not bad, bad
assert torch.equal(made[0][1], made[1][1]) and made[0][1].abs().max() > 0 and all(m[0].check()[0] == 0 for m in made)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("window,n_first", [(0, 0), (20, 0), (20, 4), (500, 3)])
def test_positions_past_the_table(window, n_first):
    # the table holds 64 rows; a query past it sees those of them that its mask leaves, and the rest are missing
    queries = [(0, 63), (0, 64), (0, 70), (0, 83), (0, 84), (0, 95), (1, 100), (0, 1000), (1, 30), (0, 300000)]
    c = Case([64, 50], page=32, window=window, n_first=n_first, lo=[0, 9], queries=queries, seed=43)
    c.run(flags=c.b.FLAG_BAD_PAGE).check()
    # a first position at the table's end and past it: no row that the table holds is seen
    d = Case([64, 64], page=32, window=window, n_first=n_first, lo=[64, 70], queries=[(0, 64), (0, 90), (1, 90), (1, 69)], seed=44)
    d.run(flags=d.b.FLAG_BAD_PAGE).check()
    assert (d.out == 0).all()


@pytest.mark.parametrize("fmt,page", [("bf16", 4), ("fp8", 4), ("fp4", 4), ("fp8", 1), ("fp4", 2), ("bf16", 4096), ("fp8", 4096),
                                      ("fp4", 4096)])
def test_small_and_large_pages(fmt, page):
    Case([333, 1, 140], fmt=fmt, page=page, seed=page + 45).run().check()
    Case([300, 77], fmt=fmt, page=page, per=2, window=90, n_first=5, lo=[3, 0], seed=page + 46).run().check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_dense_prompt_chunk(fmt):
    # every token of a chunk over a prefix is a query and sees all rows up to its own: more tiles than two a CTA
    lens, per = [333, 210, 128], [130, 90, 60]
    queries = [(b, n - k + i) for b, (n, k) in enumerate(zip(lens, per)) for i in range(k)]
    c = Case(lens, fmt=fmt, page=32, lo=[0, 5, 0], queries=queries, seed=47).run()
    pick = sorted({*range(0, len(queries), 9), 129, 130, 219, 220, len(queries) - 1})
    c.out, c.lse, c.q = c.out[pick], c.lse[pick], c.q[pick]
    c.seq, c.pos = [c.seq[i] for i in pick], [c.pos[i] for i in pick]
    c.check()


def test_dense_prompt_chunk_from_an_empty_cache():
    # the first chunk of a prompt: query i sees i + 1 rows
    c = Case([200, 1, 131], page=16, queries=[(b, t) for b, n in enumerate([200, 1, 131]) for t in range(n)], seed=48).run()
    pick = [0, 1, 2, 63, 64, 127, 128, 129, 199, 200, 201, 202, 328, 329, 330, 331]
    c.out, c.lse, c.q = c.out[pick], c.lse[pick], c.q[pick]
    c.seq, c.pos = [c.seq[i] for i in pick], [c.pos[i] for i in pick]
    c.check()


@pytest.mark.parametrize("fmt,page", [("bf16", 4096), ("fp8", 64)])
def test_the_last_rows_of_the_largest_table(fmt, page):
    # 2^30 rows a sequence: positions, chunks and columns at the end of 32 bits
    from compressed_sparse_attention_gb300 import binding
    end, cols = 2 ** 30, 2 ** 30 // page
    n = -(-400 // page) + 1
    # the window starts 400 rows before the end; the first tokens lie right behind lo
    lens, lo = [1], [end - 300]
    c = Case(lens, fmt=fmt, page=page, window=150, n_first=5, lo=lo, queries=[(0, end - 1), (0, end - 140), (0, end - 300)],
             seed=49, spare=n + 1)
    c.table = torch.full((1, cols), -1, dtype=torch.int32, device=DEV)
    c.table[0, cols - n:] = torch.arange(n, dtype=torch.int32)
    c.kv = c.ctx.paged_kv(c.codes, c.table, c.scales)
    c.table_rows = [c.table[0].tolist()]
    c.run().check()
    c.window = 0  # every row from lo on
    c.run().check()
    c.pos = [end, end + 7, end - 2]
    c.pos_d.copy_(torch.tensor(c.pos))
    c.run(flags=binding.FLAG_BAD_PAGE).check()


def test_one_position_asked_for_by_several_queries():
    Case([900, 40], page=16, queries=[(0, 899), (1, 39), (0, 899), (0, 899), (1, 39)], seed=50).run().check()


@pytest.mark.parametrize("power", [80, -80])
def test_rows_far_from_unit_size(power):
    # weights reach 2^32 before a reference moves: 600 rows of size 4 sum to 2^(80 + 2 + 32 + 10) at most
    c = Case([600, 200, 3], page=16, seed=51, q_scale=30.0)
    c.codes *= 2.0 ** power
    c.q *= 2.0 ** -power
    c.run().check()
