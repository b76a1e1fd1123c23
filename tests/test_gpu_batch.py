"""csa2_batch_tables, csa2_query_groups and csa2_append_slots against plain
restatements with Python lists (whole numbers, equal) and, for the stored rows,
csa2_append_paged's bits and a 64-bit rotation."""
import random

import pytest
import torch

from gpu_common import context, require_gpu
from paged_common import DIM, FMT_NAMES, U16, U32, layer_turned, page_values, random_pages

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD_PAGE, BAD_SEQ, BATCH_FULL, BAD_QUERY = 0x40, 0x100, 0x200, 0x20


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


# ---------------------------------------------------------------- tables

class Pool:
    def __init__(self, lens, page=16, width=None, seed=0, extra_cols=0):
        require_gpu()
        self.ctx, self.page = context(), page
        rng = random.Random(seed)
        counts = [-(-n // page) for n in lens]
        width = width or max(1, max(counts))
        self.n_pages = sum(counts) + 3
        free = list(range(self.n_pages))
        rng.shuffle(free)
        # behind a sequence's last page the pool's row may hold anything: it is not copied
        self.rows = [[free.pop() for _ in range(c)] + [-1] * (width - c) for c in counts]
        self.lens = list(lens)
        full = torch.full((len(lens), width + extra_cols), 5, dtype=torch.int32)
        full[:, :width] = torch.tensor(self.rows, dtype=torch.int32)
        self.table = full.to(DEV)[:, :width]
        self.seq_len = i64(lens)
        self.ref = torch.ones(self.n_pages, dtype=torch.int32, device=DEV)
        self.pool = self.ctx.page_pool(self.table, self.seq_len, self.ref, page)

    def plain(self, seqs, n_new, max_tokens):
        page, flags = self.page, 0
        width = len(self.rows[0])
        table, off, first, tok = [], [0], [], []
        full = False
        for r, (b, k) in enumerate(zip(seqs, n_new)):
            ok = 0 <= b < len(self.lens) and 0 <= k <= self.lens[b] <= width * page
            if not ok:
                flags |= BAD_SEQ if b != -1 else 0
                table.append([-1] * width)
                first.append(0)
                off.append(off[-1])
                continue
            used = -(-self.lens[b] // page)
            table.append(self.rows[b][:used] + [-1] * (width - used))
            first.append(self.lens[b] - k)
            if not full and len(tok) + k > max_tokens:
                full = True
                flags |= BATCH_FULL
            if not full:
                for p in range(self.lens[b] - k, self.lens[b]):
                    g = self.rows[b][p // page]
                    there = 0 <= g < self.n_pages
                    flags |= 0 if there else BAD_PAGE
                    tok.append((r, p, g * page + p % page if there else -1))
            off.append(len(tok))
        tok += [(-1, -1, -1)] * (max_tokens - len(tok))
        return table, off, first, tok, flags

    def check(self, seqs, n_new, max_tokens, extra_cols=0, seqs_d=None):
        n, width = len(seqs), len(self.rows[0])
        table = torch.full((n, width + extra_cols), 77, dtype=torch.int32, device=DEV)
        off, first = torch.full((n + 1,), 77, device=DEV), torch.full((n,), 77, device=DEV)
        req = torch.full((max_tokens,), 77, dtype=torch.int32, device=DEV)
        pos, slot = torch.full((max_tokens,), 77, device=DEV), torch.full((max_tokens,), 77, device=DEV)
        self.ctx.batch_tables(self.pool, i32(seqs) if seqs_d is None else seqs_d, i64(n_new), table[:, :width], off, first,
                              req, pos, slot)
        got, _ = self.ctx.check()
        want = self.plain(seqs, n_new, max_tokens)
        assert got == want[4], f"flags {got:#x}, not {want[4]:#x}"
        assert table[:, :width].tolist() == want[0]
        assert (table[:, width:] == 77).all()
        assert off.tolist() == want[1] and first.tolist() == want[2]
        assert list(zip(req.tolist(), pos.tolist(), slot.tolist())) == want[3]


@pytest.mark.parametrize("page", [1, 8, 16, 256, 4096])
def test_tables_of_a_decode_step(page):
    p = Pool([5, 16, 17, 300, 1, 32], page=page)
    p.check([3, 0, 5, 2], [1, 1, 1, 1], 4)
    p.check([3, 0, 5, 2], [1, 1, 1, 1], 9)


def test_tables_of_one_request():
    p = Pool([5])
    p.check([0], [1], 1)
    p.check([0], [5], 5)
    p.check([0], [0], 0)
    p.check([0], [0], 3)
    p.check([-1], [9], 3)


@pytest.mark.parametrize("n", [2, 255, 256, 257, 1023, 1024, 1025, 2500])
def test_tables_of_many_requests(n):
    rng = random.Random(n)
    p = Pool([rng.randint(1, 200) for _ in range(n + 3)], seed=n, extra_cols=3)
    seqs = rng.sample(range(n + 3), n)
    new = [min(p.lens[b], rng.choice([0, 1, 1, 1, rng.randint(1, 200)])) for b in seqs]
    p.check(seqs, new, sum(new) + rng.choice([0, 1, 1000]), extra_cols=5)


def test_tables_of_empty_sequences_and_padding_requests():
    p = Pool([0, 7, 0, 16, 33])
    p.check([0, -1, 1, 2, 3, -1, 4, -1], [0, 5, 7, 0, 16, 0, 1, -4], 40)


def test_a_sequence_named_twice():
    p = Pool([20, 30])
    p.check([1, 0, 1, 1], [2, 3, 30, 1], 40)


def test_tables_of_bad_requests():
    p = Pool([20, 30, 10])
    p.check([0, 3, 1, -2, 2, 1], [1, 1, 31, 1, -1, 4], 20)


@pytest.mark.parametrize("max_tokens", [0, 1, 9, 10, 11, 39, 40])
def test_requests_past_the_capacity_have_no_tokens(max_tokens):
    p = Pool([20, 30, 10, 15])
    p.check([0, 1, 2, 3], [10, 0, 10, 15], max_tokens)


def test_capacity_ends_in_a_later_part_of_the_requests():
    rng = random.Random(1)
    p = Pool([rng.randint(1, 9) for _ in range(3000)], seed=2)
    new = list(p.lens)
    p.check(list(range(3000)), new, sum(new[:1500]) + 1)
    p.check(list(range(3000)), new, sum(new[:1024]))
    p.check(list(range(3000)), new, sum(new[:2048]) - 1)


def test_tables_with_missing_pages():
    p = Pool([64, 64])
    p.rows[1][2], p.rows[0][1] = -1, p.n_pages + 4
    p.table.copy_(i32(p.rows))
    p.check([0, 1], [64, 64], 130)


def test_a_length_past_the_table():
    p = Pool([64, 64])
    p.lens[1] = 65
    p.seq_len.copy_(i64(p.lens))
    p.check([0, 1], [1, 1], 3)


def test_wide_tables():
    p = Pool([5000, 1, 4096], page=1, width=5003)
    p.check([2, 0, 1], [4, 4500, 1], 4600)


def test_no_requests():
    p = Pool([5])
    off = torch.full((1,), 77, device=DEV)
    req, pos, slot = torch.full((3,), 7, dtype=torch.int32, device=DEV), torch.full((3,), 7, device=DEV), torch.full((3,), 7, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    p.ctx.batch_tables(p.pool, none.int(), none, torch.empty((0, 1), dtype=torch.int32, device=DEV), off, none.clone(), req, pos, slot)
    assert off.tolist() == [0] and req.tolist() == pos.tolist() == slot.tolist() == [-1] * 3


def test_a_captured_step_follows_the_pool():
    p = Pool([20, 30, 10])
    seqs, new = i32([2, 0]), i64([1, 1])
    table, off, first = torch.zeros((2, 2), dtype=torch.int32, device=DEV), i64([0] * 3), i64([0] * 2)
    req, pos, slot = i32([0] * 4), i64([0] * 4), i64([0] * 4)
    call = p.ctx.prepare_batch_tables(p.pool, seqs, new, table, off, first, req, pos, slot)
    call.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    p.lens[2], p.lens[0] = 13, 25
    p.seq_len.copy_(i64(p.lens))
    new.copy_(i64([3, 1]))
    g.replay()
    want = p.plain([2, 0], [3, 1], 4)
    assert table.tolist() == want[0] and off.tolist() == want[1] and first.tolist() == want[2]
    assert list(zip(req.tolist(), pos.tolist(), slot.tolist())) == want[3]


def test_tables_refusals():
    p = Pool([20, 30])
    b = __import__("compressed_sparse_attention_gb300.binding", fromlist=["x"])
    def call(**kw):
        a = dict(seqs=i32([0, 1]), n_new=i64([1, 1]), table=torch.zeros((2, 2), dtype=torch.int32, device=DEV), tok_off=i64([0] * 3),
                 first_pos=i64([0] * 2), req_of_tok=i32([0] * 4), tok_pos=i64([0] * 4), tok_slot=i64([0] * 4))
        a.update(kw)
        p.ctx.batch_tables(p.pool, *a.values())
    call()
    for kw in (dict(seqs=i64([0, 1])), dict(n_new=i32([1, 1])), dict(table=torch.zeros((2, 3), dtype=torch.int32, device=DEV)),
               dict(table=torch.zeros((2, 2), dtype=torch.int64, device=DEV)), dict(tok_off=i64([0] * 2)), dict(first_pos=i64([0] * 3)),
               dict(req_of_tok=i32([0] * 5)), dict(tok_pos=i32([0] * 4)), dict(tok_slot=torch.zeros(4, dtype=torch.int64)),
               dict(tok_off=None), dict(first_pos=None), dict(table=None)):
        with pytest.raises((TypeError, ValueError, AttributeError, b.Csa2Error)):
            call(**kw)


# ---------------------------------------------------------------- groups

def plain_groups(rows, page, n_pages, q_pos, seq_of_q, min_shared):
    columns, n = -(-min_shared // page), len(q_pos)
    width = len(rows[0])

    def row(i):
        return rows[seq_of_q[i]] if 0 <= seq_of_q[i] < len(rows) and q_pos[i] >= 0 else None

    def whole(i):
        return 0 if row(i) is None else min((q_pos[i] + 1) // page, width)

    lead, low = [], {}
    for i in range(n):
        key = row(i)[columns - 1] if columns <= whole(i) else -1
        lead.append(low.setdefault(key, i) if 0 <= key < n_pages else i)
    order, head, shared = [], [], []
    for g in range(n):
        mine = [i for i in range(n) if lead[i] == g]
        run = 0
        if len(mine) > 1:
            while (all(run < whole(i) for i in mine) and 0 <= row(g)[run] < n_pages and all(row(i)[run] == row(g)[run] for i in mine)):
                run += 1
        for j, i in enumerate(mine):
            head.append(len(order) - j)
            order.append(i)
            shared.append(run * page if j == 0 else 0)
    return order, head, shared, sum(1 for k, h in enumerate(head) if h == k)


def check_groups(rows, page, n_pages, q_pos, seq_of_q, min_shared, flags=0, extra_cols=0):
    require_gpu()
    ctx = context()
    full = torch.full((len(rows), len(rows[0]) + extra_cols), 3, dtype=torch.int32)
    full[:, :len(rows[0])] = torch.tensor(rows, dtype=torch.int32)
    table = full.to(DEV)[:, :len(rows[0])]
    n = len(q_pos)
    order, head, shared, groups = i32([-7] * n), i32([-7] * n), i64([-7] * n), i32([-7])
    ctx.query_groups(table, page, n_pages, i64(q_pos), i32(seq_of_q), min_shared, order, head, shared, groups)
    got, _ = ctx.check()
    assert got == flags
    want = plain_groups(rows, page, n_pages, q_pos, seq_of_q, min_shared)
    assert order.tolist() == want[0]
    assert head.tolist() == want[1]
    assert shared.tolist() == want[2]
    assert groups.tolist() == [want[3]]


def forked(n, docs, page, width, seed, least=1):
    """Rows of n sequences that share runs of pages of `docs` documents, and their lengths."""
    rng = random.Random(seed)
    free = iter(rng.sample(range(4 * n * width + 4 * docs * width), 2 * n * width + 2 * docs * width))
    first = [[next(free) for _ in range(width)] for _ in range(docs)]
    rows, lens = [], []
    for _ in range(n):
        k = rng.randint(1, width)
        share = min(k, rng.randint(0, width))
        rows.append(rng.choice(first)[:share] + [next(free) for _ in range(k - share)] + [-1] * (width - k))
        lens.append((k - 1) * page + rng.randint(1, page))
    return rows, lens, 4 * n * width + 4 * docs * width


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 255, 256, 257, 1000, 2048, 4096])
@pytest.mark.parametrize("min_shared", [1, 33])
def test_groups_of_many_queries(n, min_shared):
    rows, lens, n_pages = forked(n, max(1, n // 7), 16, 9, n)
    check_groups(rows, 16, n_pages, [m - 1 for m in lens], list(range(n)), min_shared, extra_cols=2)


@pytest.mark.parametrize("page", [1, 8, 64, 4096])
@pytest.mark.parametrize("min_shared", [1, 2, 64, 65, 4097, 1 << 50])
def test_groups_by_page_size_and_length(page, min_shared):
    rows, lens, n_pages = forked(60, 4, page, 80, page)
    check_groups(rows, page, n_pages, [m - 1 for m in lens], list(range(60)), min_shared)


def test_one_group_of_all():
    n = 4096
    rows = [[5, 6, 7, 100 + i] for i in range(n)]
    check_groups(rows, 16, 100 + n, [16 * 3 + i % 17 for i in range(n)], list(range(n)), 20)


def test_no_groups():
    check_groups([[i, 50 + i] for i in range(40)], 16, 100, [31] * 40, list(range(40)), 1)


def test_queries_of_one_sequence_are_a_group():
    check_groups([[4, 5, 6], [4, 5, 7]], 16, 10, [47, 30, 31, 15, 40, 14], [0, 0, 1, 1, 0, 0], 1)


def test_rows_that_share_a_column_but_not_the_ones_before():
    check_groups([[1, 9, 3], [2, 9, 3], [1, 9, 4]], 16, 20, [47, 47, 47], [0, 1, 2], 32)


def test_missing_pages_end_a_common_run():
    rows = [[1, 2, -1, 4], [1, 2, -1, 4], [1, 2, 77, 4], [1, 2, 77, 5]]
    check_groups(rows, 16, 50, [63] * 4, [0, 1, 2, 3], 1)
    check_groups(rows, 16, 50, [63] * 4, [0, 1, 2, 3], 40)
    check_groups(rows, 16, 50, [63] * 5, [0, 0, 2, 2, 2], 1)


def test_groups_of_padding_and_bad_queries():
    check_groups([[1, 2], [1, 3]], 16, 10, [20, -1, 25, 31, 5], [0, 1, -1, 1, -1], 1)
    check_groups([[1, 2], [1, 3]], 16, 10, [20, -2, 25, 31], [0, 1, 7, 1], 1, flags=BAD_QUERY)


def test_lengths_bound_the_common_run():
    check_groups([[1, 2, 3, 4]] * 5, 16, 10, [63, 62, 47, 46, 15], [0, 1, 2, 3, 4], 16)


def test_positions_past_the_table_in_groups():
    check_groups([[1, 2, 3, 4]] * 4, 16, 10, [1 << 40, 63, 1000, (1 << 63) - 1], [0, 1, 2, 3], 16)


def test_groups_on_another_stream_and_captured():
    require_gpu()
    ctx = context()
    rows, lens, n_pages = forked(100, 5, 16, 9, 77)
    table, seq, pos = i32(rows), i32(list(range(100))), i64([m - 1 for m in lens])
    out = [i32([0] * 100), i32([0] * 100), i64([0] * 100), i32([0])]
    call = ctx.prepare_query_groups(table, 16, n_pages, pos, seq, 16, *out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call.run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    pos.sub_(20).clamp_(min=-1)
    g.replay()
    want = plain_groups(rows, 16, n_pages, pos.tolist(), list(range(100)), 16)
    assert [o.tolist() for o in out] == [want[0], want[1], want[2], [want[3]]]


def test_groups_refusals():
    require_gpu()
    ctx = context()
    b = __import__("compressed_sparse_attention_gb300.binding", fromlist=["x"])
    def call(**kw):
        a = dict(table=i32([[1, 2], [1, 3]]), page_size=16, n_pages=9, q_pos=i64([20, 20]), seq_of_q=i32([0, 1]), min_shared=1,
                 order=i32([0, 0]), head=i32([0, 0]), shared=i64([0, 0]), n_groups=None)
        a.update(kw)
        ctx.query_groups(*a.values())
    call()
    big = 4097
    for kw in (dict(page_size=3), dict(page_size=0), dict(n_pages=0), dict(min_shared=0), dict(min_shared=-4), dict(q_pos=i32([20, 20])),
               dict(seq_of_q=i64([0, 1])), dict(order=i64([0, 0])), dict(head=i32([0])), dict(shared=i32([0, 0])),
               dict(table=i64([[1, 2], [1, 3]])), dict(n_groups=i64([0])), dict(order=None), dict(shared=None), dict(seq_of_q=None),
               dict(q_pos=i64([0] * big), seq_of_q=i32([0] * big), order=i32([0] * big), head=i32([0] * big), shared=i64([0] * big))):
        with pytest.raises((TypeError, ValueError, AttributeError, b.Csa2Error)):
            call(**kw)


# ---------------------------------------------------------------- rows by slot

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,n", [(1, 1), (16, 7), (64, 33), (256, 130)])
def test_slots_hold_what_append_paged_stores(fmt, dtype, page, n):
    require_gpu()
    ctx = context(kv_format=fmt)
    n_pages = 2 * (-(-n // page)) + 3
    codes, scales = random_pages(FMT_NAMES[fmt], n_pages, page, n, DEV)
    one, one_s = codes.clone(), None if scales is None else scales.clone()
    rng = random.Random(n)
    k = -(-(n + 3) // page)
    row = rng.sample(range(n_pages), k)
    rows = torch.randn((n, DIM), generator=torch.Generator().manual_seed(n)).to(dtype).to(DEV)
    ctx.append_paged(ctx.paged_kv(codes, i32([row]), scales), rows, i64([0, n]), i64([3]))
    # the same rows in another order
    perm = rng.sample(range(n), n)
    pos = [3 + i for i in perm]
    slots = [row[p // page] * page + p % page for p in pos]
    ctx.append_slots(ctx.paged_kv(one, None, one_s), rows[perm], i64(pos), i64(slots))
    assert ctx.check()[0] == 0
    assert torch.equal(codes.view(torch.uint8), one.view(torch.uint8))
    assert scales is None or torch.equal(scales, one_s)


def test_slots_against_the_rotation():
    require_gpu()
    ctx = context()
    codes = torch.zeros((9, 16, DIM), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(5)
    rows = torch.randn((40, DIM), generator=g)
    pos = torch.randint(0, 1 << 21, (40,), generator=g)
    slots = torch.randperm(9 * 16, generator=g)[:40]
    ctx.append_slots(ctx.paged_kv(codes), rows.to(DEV), pos.to(DEV), slots.to(DEV))
    want = torch.zeros((9 * 16, DIM), dtype=torch.float64)
    want[slots] = layer_turned(rows.double(), pos[:, None], ctx.cfg)
    got = codes.view(-1, DIM).double().cpu()
    # bf16 of an fp32 rotation: half a step, and of the pair's size the cosine's and
    # sine's error (2^-23 each, the products' and the sum's roundings 3 U32) and the
    # angle's (2^21 radians in double precision reduced with a relative 2^-53: 2^-31)
    size = rows.double().abs().reshape(40, -1, 2).sum(-1).repeat_interleave(2, -1)
    bound = torch.zeros_like(want)
    bound[slots] = U16 * want[slots].abs() + size * (2 * 2.0 ** -23 + 3 * U32 + 2.0 ** -31) * (1 + U16)
    assert ((got - want).abs() <= bound).all()


def test_rows_without_positions_are_not_rotated():
    require_gpu()
    ctx = context()
    codes = torch.zeros((2, 4, DIM), dtype=torch.bfloat16, device=DEV)
    rows = torch.randn((3, DIM), device=DEV).to(torch.bfloat16)
    ctx.append_slots(ctx.paged_kv(codes), rows, None, i64([7, 0, 3]))
    assert torch.equal(codes.view(-1, DIM)[[7, 0, 3]], rows)
    assert (codes.view(-1, DIM)[[1, 2, 4, 5, 6]] == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_padding_and_bad_slots(fmt):
    require_gpu()
    ctx = context(kv_format=fmt)
    codes, scales = random_pages(FMT_NAMES[fmt], 5, 8, 1, DEV)
    was, was_s = codes.clone(), None if scales is None else scales.clone()
    rows = torch.randn((4, DIM), device=DEV)
    kv = ctx.paged_kv(codes, None, scales)
    ctx.append_slots(kv, rows, i64([-1, -5, 7, 3]), i64([-1] * 4))
    assert ctx.check()[0] == 0
    for pos, slot in ((0, 40), (0, -2), (0, 1 << 50), (-1, 3), (0, -(1 << 60))):
        ctx.append_slots(kv, rows[:1], i64([pos]), i64([slot]))
        assert ctx.check()[0] == BAD_PAGE
    assert torch.equal(codes.view(torch.uint8), was.view(torch.uint8)) and (scales is None or torch.equal(scales, was_s))


def test_slots_of_strided_pages_past_32_bits():
    require_gpu()
    ctx = context()
    all_layers = torch.zeros((70000, 2, 32, DIM), dtype=torch.bfloat16, device=DEV)
    codes = all_layers[:, 1]
    rows = torch.randn((2, DIM), device=DEV).to(torch.bfloat16)
    ctx.append_slots(ctx.paged_kv(codes), rows, None, i64([69999 * 32 + 31, 5]))
    assert ctx.check()[0] == 0
    assert torch.equal(codes[69999, 31], rows[0]) and torch.equal(codes[0, 5], rows[1])
    assert int((all_layers != 0).any(-1).sum()) == 2


def test_slots_refusals():
    require_gpu()
    ctx = context()
    b = __import__("compressed_sparse_attention_gb300.binding", fromlist=["x"])
    codes = torch.zeros((2, 4, DIM), dtype=torch.bfloat16, device=DEV)
    rows = torch.randn((3, DIM), device=DEV).to(torch.bfloat16)
    def call(**kw):
        a = dict(kv=ctx.paged_kv(codes), rows=rows, pos=i64([1, 2, 3]), slots=i64([0, 1, 2]))
        a.update(kw)
        ctx.append_slots(*a.values())
    call()
    for kw in (dict(rows=rows.half()), dict(rows=rows[:, :256].contiguous()), dict(pos=i32([1, 2, 3])), dict(slots=i32([1, 2, 3])),
               dict(slots=i64([1, 2])), dict(pos=i64([1])), dict(slots=None), dict(rows=rows.cpu())):
        with pytest.raises((TypeError, ValueError, b.Csa2Error)):
            call(**kw)
    ctx.append_slots(ctx.paged_kv(codes), rows[:0], i64([]), i64([]))
    assert ctx.last_launch_count == 0


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_a_serving_step_from_lengths_alone(fmt):
    """Requests forked from two prompts decode for some steps: pages, tables,
    slots, groups and attention all made on the device, against the packed path
    (append_paged by the pool's own table, attend_paged query by query)."""
    require_gpu()
    from compressed_sparse_attention_gb300 import binding
    from paged_common import check_attend
    ctx, page, n_seq, width = context(kv_format=fmt), 16, 8, 24
    f = FMT_NAMES[fmt]
    n_pages = 140
    codes, scales = random_pages(f, n_pages, page, 3, DEV)
    table = torch.full((n_seq, width), -1, dtype=torch.int32, device=DEV)
    seq_len, ref = i64([0] * n_seq), i32([0] * n_pages)
    pool = ctx.page_pool(table, seq_len, ref, page)
    ws = binding.workspace(ctx.pages_workspace_size(pool), DEV)
    arrays = [codes] + ([] if scales is None else [scales])
    ctx.pages_extend(pool, i32([0, 4]), i64([150, 203]), ws)
    ctx.pages_fork(pool, i32([0, 0, 0, 4, 4]), i32([1, 2, 3, 5, 6]), arrays, ws)
    seqs = i32([0, 1, 2, 4, 5, 6, 3, -1])  # the last a padding request
    n_req, cap = 8, 16
    batch = dict(table=torch.empty((n_req, width), dtype=torch.int32, device=DEV), tok_off=i64([0] * 9), first_pos=i64([0] * 8),
                 req_of_tok=i32([0] * cap), tok_pos=i64([0] * cap), tok_slot=i64([0] * cap))
    order, head, shared = i32([0] * cap), i32([0] * cap), i64([0] * cap)
    kv = ctx.paged_kv(codes, batch["table"], scales)
    q = torch.randn((cap, 64, DIM), device=DEV).to(torch.bfloat16)
    rows = torch.randn((cap, DIM), device=DEV).to(torch.bfloat16)
    sink = torch.randn(64, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((cap, 64), device=DEV)
    aws = binding.workspace(ctx.attend_shared_workspace_size(cap), DEV)
    grow = i64([2, 1, 1, 1, 2, 1, 1, 0])
    new_len = torch.zeros(8, dtype=torch.int64, device=DEV)

    def step():
        new_len.copy_(torch.where(seqs >= 0, seq_len[seqs.clamp_min(0).long()] + grow, 0))
        ctx.pages_extend(pool, seqs, new_len, ws)
        ctx.batch_tables(pool, seqs, grow, **batch)
        ctx.append_slots(kv, rows, batch["tok_pos"], batch["tok_slot"])
        ctx.query_groups(batch["table"], page, n_pages, batch["tok_pos"], batch["req_of_tok"], 32, order, head, shared)
        ctx.attend_shared(kv, q, batch["tok_pos"], batch["req_of_tok"], order, head, shared, out, aws, sink=sink, lse=lse)

    step()
    assert ctx.check()[0] == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        rows.normal_()
        q.normal_()
        g.replay()
    assert ctx.check()[0] == 0
    torch.cuda.synchronize()
    used = int(batch["tok_off"][-1])
    assert used == 9 and shared.tolist()[0] == 144
    t = batch["table"].tolist()
    check_attend(out[:used], lse[:used], page_values(codes, scales, f), t, page, q[:used], batch["tok_pos"].tolist()[:used],
                 batch["req_of_tok"].tolist()[:used], None, 0, 0, sink, ctx.cfg)
    # the packed append stores the same bytes
    codes2, scales2 = codes.clone(), None if scales is None else scales.clone()
    ctx.append_paged(ctx.paged_kv(codes2, batch["table"], scales2), rows, batch["tok_off"], batch["first_pos"])
    assert torch.equal(codes.view(torch.uint8), codes2.view(torch.uint8))


def test_a_batchs_table_over_the_pools_is_refused():
    p = Pool([20, 30, 40])
    b = __import__("compressed_sparse_attention_gb300.binding", fromlist=["x"])
    n, w = 2, len(p.rows[0])
    both = torch.zeros((6, w), dtype=torch.int32, device=DEV)
    both[:3] = p.table
    pool = p.ctx.page_pool(both[:3], p.seq_len, p.ref, p.page)
    rest = (i64([0] * 3), i64([0] * 2), i32([0] * 4), i64([0] * 4), i64([0] * 4))
    for at in (0, 1, 2):
        with pytest.raises(b.Csa2Error, match="overlaps"):
            p.ctx.batch_tables(pool, i32([0, 1]), i64([1, 1]), both[at:at + 2], *rest)
    p.ctx.batch_tables(pool, i32([0, 1]), i64([1, 1]), both[3:5], *rest)
    assert p.ctx.check()[0] == 0 and both[3:5].tolist() == p.rows[:2]


def test_batch_calls_from_a_host_thread_without_cuda_calls():
    import threading
    p = Pool([20, 30, 10])
    ctx = p.ctx
    table, off, first = torch.zeros((2, 2), dtype=torch.int32, device=DEV), i64([0] * 3), i64([0] * 2)
    req, pos, slot = i32([0] * 4), i64([0] * 4), i64([0] * 4)
    order, head, shared = i32([0] * 4), i32([0] * 4), i64([0] * 4)
    pages = torch.zeros((p.n_pages, 16, DIM), dtype=torch.bfloat16, device=DEV)
    rows = torch.randn((4, DIM), device=DEV).to(torch.bfloat16)
    calls = [ctx.prepare_batch_tables(p.pool, i32([2, 0]), i64([1, 2]), table, off, first, req, pos, slot),
             ctx.prepare_append_slots(ctx.paged_kv(pages), rows, pos, slot),
             ctx.prepare_query_groups(table, 16, p.n_pages, pos, req, 1, order, head, shared)]
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            for c in calls:
                c.run()
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    want = p.plain([2, 0], [1, 2], 4)
    assert list(zip(req.tolist(), pos.tolist(), slot.tolist())) == want[3]
    assert order.tolist() == [0, 1, 2, 3] and head.tolist() == [0, 1, 1, 3] and shared.tolist() == [0, 16, 0, 0]
    assert int((pages != 0).any(-1).sum()) == 3


@pytest.mark.parametrize("n", [1, 5, 40])
def test_two_streams_at_once(n):
    """Each stream its own context and outputs, one table read by both."""
    require_gpu()
    from compressed_sparse_attention_gb300 import binding
    rows, lens, n_pages = forked(50, 3, 16, 9, n)
    table, seq, pos = i32(rows), i32(list(range(50))), i64([m - 1 for m in lens])
    made = []
    for _ in range(2):
        ctx = binding.Context()
        out = [i32([0] * 50), i32([0] * 50), i64([0] * 50), i32([0])]
        made.append((ctx.prepare_query_groups(table, 16, n_pages, pos, seq, n, *out), out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, _, s in made:
            with torch.cuda.stream(s):
                call.run()
    torch.cuda.synchronize()
    want = plain_groups(rows, 16, n_pages, pos.tolist(), list(range(50)), n)
    for _, out, _ in made:
        assert [o.tolist() for o in out] == [want[0], want[1], want[2], [want[3]]]
