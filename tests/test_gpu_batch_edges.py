"""csa2_batch_tables, csa2_query_groups and csa2_append_slots at the ends of
their ranges: nothing to do, padded batches, many requests."""
import random

import pytest
import torch

from gpu_common import context, require_gpu
from test_gpu_batch import BAD_SEQ, BATCH_FULL, DEV, Pool, i32, i64

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- groups

def groups_of_nothing(ctx, n_groups):
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    return ctx.prepare_query_groups(i32([[1, 2]]), 16, 9, none, none.int(), 1, none.int(), none.int(), none.clone(), n_groups)


def test_no_queries_are_no_groups():
    require_gpu()
    ctx = context()
    n_groups = i32([7, 7])
    groups_of_nothing(ctx, n_groups[:1]).run()
    assert ctx.last_launch_count == 0
    assert ctx.check()[0] == 0
    assert n_groups.tolist() == [0, 7]
    groups_of_nothing(ctx, None).run()


def test_no_queries_are_no_groups_on_a_stream_and_in_a_graph():
    require_gpu()
    ctx = context()
    n_groups = i32([7])
    call = groups_of_nothing(ctx, n_groups)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call.run()
    torch.cuda.current_stream().wait_stream(s)
    assert n_groups.tolist() == [0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    n_groups.fill_(9)
    g.replay()
    assert n_groups.tolist() == [0]


# ---------------------------------------------------------------- tables

def plain_tables(lens, seqs, n_new, max_tokens):
    """Offsets, first positions and (request, position) of each place, on the host with tensors."""
    ok = (seqs >= 0) & (seqs < lens.numel())
    length = torch.where(ok, lens[seqs.clamp(0, lens.numel() - 1)], 0)
    ok &= (n_new >= 0) & (n_new <= length)
    length, new = torch.where(ok, length, 0), torch.where(ok, n_new, 0)
    first = length - new
    end = torch.cumsum(new, 0)
    past = torch.nonzero(end > max_tokens)
    if past.numel():  # from the first that does not fit on: none
        new[int(past[0]):] = 0
    off = torch.cat((torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)))
    used = int(off[-1])
    req = torch.repeat_interleave(torch.arange(seqs.numel()), new)
    pos = first[req] + torch.arange(used) - off[req]
    pad = torch.full((max_tokens - used,), -1)
    flags = (0 if bool((ok | (seqs == -1)).all()) else BAD_SEQ) | (BATCH_FULL if past.numel() else 0)
    return off, first, torch.cat((req, pad)), torch.cat((pos, pad)), flags


@pytest.mark.parametrize("n,per,spare,launches", [
    (1024, 30, 0, 1), (1025, 3, 5000, 1), (3000, 40, -30000, 1), (5000, 3, 1 << 20, 2), (5000, 300, 12345, 2),
    (20000, 40, -200000, 2), (70000, 1, 0, 1), (70000, 2, 100000, 2), (1 << 20, 1, 3, 2)])
def test_tables_of_so_many_requests(n, per, spare, launches):
    """Batches around the limit of what every token CTA scans for itself: every output."""
    require_gpu()
    ctx, page = context(), 64
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 2 * per + 3, (n + 5,), generator=g)
    width = -(-(2 * per + 3) // page)
    table = torch.randperm((n + 5) * width, generator=g).reshape(n + 5, width).int()
    seqs = torch.randperm(n + 5, generator=g)[:n]
    n_new = torch.minimum(lens[seqs], torch.randint(0, 2 * per + 1, (n,), generator=g))
    seqs[torch.randint(0, n, (n // 50,), generator=g)] = -1
    if n % 2 == 0:  # some that cannot be carried out
        seqs[n // 2], n_new[n // 3] = n + 5, -4
    max_tokens = max(0, int(n_new.clamp_min(0).sum()) + spare)
    off, first, req, pos, flags = plain_tables(lens, seqs, n_new, max_tokens)
    d = [x.to(DEV) for x in (table, lens, seqs.int(), n_new)]
    pool = ctx.page_pool(d[0], d[1], torch.ones((n + 5) * width, dtype=torch.int32, device=DEV), page)
    got = dict(table=torch.full((n, width), 77, dtype=torch.int32, device=DEV), tok_off=torch.full((n + 1,), 77, device=DEV),
               first_pos=torch.full((n,), 77, device=DEV), req_of_tok=torch.full((max_tokens,), 77, dtype=torch.int32, device=DEV),
               tok_pos=torch.full((max_tokens,), 77, device=DEV), tok_slot=torch.full((max_tokens,), 77, device=DEV))
    ctx.batch_tables(pool, d[2], d[3], **got)
    assert ctx.last_launch_count == launches
    assert ctx.check()[0] == flags
    assert torch.equal(got["tok_off"].cpu(), off) and torch.equal(got["first_pos"].cpu(), first)
    assert torch.equal(got["req_of_tok"].cpu().long(), req) and torch.equal(got["tok_pos"].cpu(), pos)
    c, at = req.clamp_min(0), pos.clamp_min(0)
    slot = table[seqs[c].clamp_min(0), at // page].long() * page + at % page
    assert torch.equal(got["tok_slot"].cpu(), torch.where(req >= 0, slot, -1))
    length = torch.where((seqs >= 0) & (seqs < n + 5) & (n_new >= 0), lens[seqs.clamp(0, n + 4)], 0)
    used = (length + page - 1) // page
    rows = torch.where(torch.arange(width)[None] < used[:, None], table[seqs.clamp(0, n + 4)], -1)
    assert torch.equal(got["table"].cpu(), rows)


def test_tables_of_many_requests_in_a_graph_and_again():
    # the second launch reads the offsets that the first has written, call after call
    p = Pool([random.Random(i).randint(1, 9) for i in range(2000)], seed=7)
    seqs, new = i32(list(range(2000))), i64([0] * 2000)
    tokens = 3 << 20
    off, first, table = i64([0] * 2001), i64([0] * 2000), torch.empty_like(p.table)
    req, pos, slot = (torch.zeros(tokens, dtype=t, device=DEV) for t in (torch.int32, torch.int64, torch.int64))
    call = p.ctx.prepare_batch_tables(p.pool, seqs, new, table, off, first, req, pos, slot)
    call.run()
    assert p.ctx.last_launch_count == 2
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    for part in (1, 2):
        new.copy_(i64([m // part for m in p.lens]))
        g.replay()
        want = plain_tables(torch.tensor(p.lens), torch.arange(2000), new.cpu(), tokens)
        for a, b in zip((off, first, req.long(), pos), want):
            assert torch.equal(a.cpu(), b)


def test_tables_of_many_bad_requests_record_them():
    p = Pool([4, 5])
    n = 3000
    seqs = [0, 1] * (n // 2)
    seqs[2900] = 2
    p.check(seqs, [1] * n, n)
    p.check(seqs, [1] * n, 40)


# ---------------------------------------------------------------- rows by slot

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slots_of_a_padded_batch_hold_the_packed_rows(fmt, dtype):
    """A pool's batch by its slots, codes and scales as csa2_append_paged leaves
    them; half of the places are padding, whose rows are not looked at."""
    from paged_common import FMT_NAMES, random_pages
    page = 16
    p = Pool([40, 70, 33, 16], page=page, seed=5)
    ctx = context(kv_format=fmt)
    codes, scales = random_pages(FMT_NAMES[fmt], p.n_pages, page, 6, DEV)
    mine, mine_s = codes.clone(), None if scales is None else scales.clone()
    seqs, new = i32([2, 0, -1, 3, 1]), i64([7, 1, 0, 16, 40])
    n, cap, w = 5, 128, len(p.rows[0])
    table, off, first = torch.empty((n, w), dtype=torch.int32, device=DEV), i64([0] * 6), i64([0] * 5)
    req, pos, slot = i32([0] * cap), i64([0] * cap), i64([0] * cap)
    pool = ctx.page_pool(p.table, p.seq_len, p.ref, page)
    ctx.batch_tables(pool, seqs, new, table, off, first, req, pos, slot)
    rows = torch.randn((cap, 512), generator=torch.Generator().manual_seed(7)).to(dtype).to(DEV)
    rows[64:] = float("nan")
    ctx.append_slots(ctx.paged_kv(mine, None, mine_s), rows, pos, slot)
    ctx.append_paged(ctx.paged_kv(codes, table, scales), rows, off, first)
    assert ctx.check()[0] == 0 and off.tolist()[-1] == 64
    assert torch.equal(codes.view(torch.uint8), mine.view(torch.uint8))
    assert scales is None or torch.equal(scales, mine_s)


# ---------------------------------------------------------------- overlaps

def test_tables_over_each_other_are_refused():
    """Every pair of an output with an input or another output, in one buffer:
    the last element of one the first of the other, and one behind the other."""
    from compressed_sparse_attention_gb300 import binding
    p = Pool([20, 30, 40, 50], page=16)
    ctx, w, n, cap = p.ctx, len(p.rows[0]), 3, 9
    size = dict(seqs=(4, n), n_new=(8, n), table=(4, n * w), tok_off=(8, n + 1), first_pos=(8, n), req_of_tok=(4, cap),
                tok_pos=(8, cap), tok_slot=(8, cap), pool_table=(4, 4 * w), seq_len=(8, 4))
    outs = ("table", "tok_off", "first_pos", "req_of_tok", "tok_pos", "tok_slot")
    values = dict(seqs=i32([1, 3, 0]), n_new=i64([2, 3, 1]), pool_table=p.table.flatten(), seq_len=p.seq_len)

    def call(at):
        """Arrays at the given byte offsets of one buffer."""
        buf = torch.zeros(1 << 14, dtype=torch.uint8, device=DEV)
        a = {}
        for k, o in at.items():
            width, count = size[k]
            a[k] = buf[o:o + width * count].view(torch.int32 if width == 4 else torch.int64)
            if k in values:
                a[k].copy_(values[k])
        pool = ctx.page_pool(a["pool_table"].view(4, w), a["seq_len"], p.ref, p.page)
        ctx.batch_tables(pool, a["seqs"], a["n_new"], a["table"].view(n, w), a["tok_off"], a["first_pos"], a["req_of_tok"],
                         a["tok_pos"], a["tok_slot"])
        return a

    apart, o = {}, 0
    for k, (width, count) in size.items():
        apart[k] = o
        o += -(-width * count // 8) * 8 + 64
    want = p.plain([1, 3, 0], [2, 3, 1], cap)
    a = call(apart)
    assert a["tok_off"].tolist() == want[1] and a["first_pos"].tolist() == want[2]
    assert list(zip(a["req_of_tok"].tolist(), a["tok_pos"].tolist(), a["tok_slot"].tolist())) == want[3]
    for x in outs:
        for y in size:
            if x == y:
                continue
            (wx, cx), (wy, cy) = size[x], size[y]
            # y's first bytes over x's last, and x's first over y's last
            for first, second, end in ((x, y, wx * cx), (y, x, wy * cy)):
                over = (end - 1) // 8 * 8
                with pytest.raises(binding.Csa2Error, match="overlap"):
                    call({**apart, first: 8192, second: 8192 + over})
                call({**apart, first: 8192, second: 8192 + over + 8})
    assert ctx.check()[0] == 0


def test_arrays_between_the_rows_of_a_table_are_taken():
    # rows of a wide buffer whose other columns hold the requests and the offsets
    from compressed_sparse_attention_gb300 import binding
    p = Pool([20, 30, 40], page=16)
    w = len(p.rows[0])
    buf = torch.zeros((4, 64), dtype=torch.int32, device=DEV)
    rest = (torch.zeros(2, dtype=torch.int64, device=DEV), i32([0] * 4), i64([0] * 4), i64([0] * 4))
    for at, good in ((0, False), (w // 2 - 1 + w % 2, False), (-(-w // 2), True), (29, True), (30, False)):
        # (the last two 64-bit places of a row and the first of the next)
        tok_off = buf.view(torch.int64).flatten()[32 + at:32 + at + 3]
        if good:
            p.ctx.batch_tables(p.pool, i32([1, 2]), i64([1, 2]), buf[1:3, :w], tok_off, *rest)
            assert tok_off.tolist() == [0, 1, 3] and buf[1:3, :w].tolist() == p.rows[1:3]
        else:
            with pytest.raises(binding.Csa2Error, match="overlap"):
                p.ctx.batch_tables(p.pool, i32([1, 2]), i64([1, 2]), buf[1:3, :w], tok_off, *rest)
    assert p.ctx.check()[0] == 0


def test_groups_over_their_queries_are_refused():
    require_gpu()
    from compressed_sparse_attention_gb300 import binding
    ctx = context()
    table = i32([[1, 2], [1, 3], [1, 2]])
    pos, seq = i64([20, 20, 31]), i32([0, 1, 2])
    order, head, shared, groups = i32([0] * 3), i32([0] * 3), i64([0] * 3), i32([0])
    good = dict(table=table, page_size=16, n_pages=9, q_pos=pos, seq_of_q=seq, min_shared=1, order=order, head=head, shared=shared,
                n_groups=groups)
    for kw in (dict(shared=pos), dict(order=seq), dict(head=seq), dict(order=head), dict(n_groups=seq[2:]), dict(n_groups=order[:1]),
               dict(order=table.flatten()[3:6]), dict(n_groups=table.flatten()[5:]), dict(q_pos=shared),
               dict(head=shared.view(torch.int32)[3:])):
        with pytest.raises(binding.Csa2Error, match="overlap"):
            ctx.query_groups(**{**good, **kw})
    ctx.query_groups(**good)
    assert ctx.check()[0] == 0 and order.tolist() == [0, 1, 2] and head.tolist() == [0, 0, 0] and shared.tolist() == [16, 0, 0]
