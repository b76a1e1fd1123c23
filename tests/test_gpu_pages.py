"""The page operations against their restatement with Python lists
(paged_common.HostPool): tables, lengths, counts, flags and page contents are
equal, value for value."""
import random

import pytest
import torch

from gpu_common import context, require_gpu
from paged_common import HostPool

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Pool:
    """A device pool beside its host restatement."""

    def __init__(self, lens, page=16, n_pages=64, cols=None, seed=0, arrays=((torch.bfloat16, 8), (torch.uint8, 16)),
                 extra_cols=0, layers=0):
        from compressed_sparse_attention_gb300 import binding
        require_gpu()
        self.ctx = context()
        rng = random.Random(seed)
        order = list(range(n_pages))
        rng.shuffle(order)
        cols = cols or max(1, max(-(-n // page) for n in lens) + 3)
        rows, ref = [], [0] * n_pages
        for n in lens:
            got = [order.pop() for _ in range(-(-n // page))]
            for g in got:
                ref[g] = 1
            rows.append(got + [-1] * (cols - len(got)))
        self.host = HostPool(rows, lens, ref, page)
        full = torch.full((len(lens), cols + extra_cols), 99, dtype=torch.int32)
        full[:, :cols] = torch.tensor(rows, dtype=torch.int32)
        self.full = full.to(DEV)
        self.table = self.full[:, :cols]
        self.seq_len = torch.tensor(lens, dtype=torch.int64, device=DEV)
        self.ref = torch.tensor(ref, dtype=torch.int32, device=DEV)
        self.arrays = []
        g = torch.Generator().manual_seed(seed)
        for dt, width in arrays:
            shape = (n_pages, layers, page, width) if layers else (n_pages, page, width)
            raw = torch.randint(0, 256, shape[:-1] + (width * torch.empty((), dtype=dt).element_size(),), generator=g,
                                dtype=torch.uint8).to(DEV)
            self.arrays.append(raw[:, -1] if layers else raw)
        self.model = [a.clone() for a in self.arrays]
        self.pool = self.ctx.page_pool(self.table, self.seq_len, self.ref, page)
        self.ws = binding.workspace(self.ctx.pages_workspace_size(self.pool), DEV)

    @staticmethod
    def ids(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=DEV)

    def do(self, name, *args, **kw):
        """The operation on the device and in the restatement, then all state compared."""
        ids = self.ids
        call = {"extend": lambda: self.ctx.pages_extend(self.pool, ids(args[0]), ids(args[1], torch.int64), self.ws),
                "fork": lambda: self.ctx.pages_fork(self.pool, ids(args[0]), ids(args[1]), self.arrays, self.ws, **kw),
                "free": lambda: self.ctx.pages_free(self.pool, ids(args[0])),
                "trim": lambda: self.ctx.pages_trim(self.pool, ids(args[0]), args[1], args[2],
                                                    None if len(args) < 4 else ids(args[3], torch.int64))}[name]
        call()
        getattr(self.host, name)(*args, **kw)
        self.compare()

    def compact(self):
        n = torch.full((1,), -5, dtype=torch.int32, device=DEV)
        self.ctx.pages_compact(self.pool, self.arrays, n, self.ws)
        assert self.host.compact() == n.item()
        self.compare()

    def compare(self):
        h = self.host
        flags, _ = self.ctx.check()
        assert flags == h.flags, f"flags 0x{flags:x}, expected 0x{h.flags:x}"
        h.flags = 0
        assert self.table.tolist() == h.table
        assert self.seq_len.tolist() == h.len
        assert self.ref.tolist() == h.ref
        assert (self.full[:, self.table.shape[1]:] == 99).all()
        old = [m.clone() for m in self.model]
        for s, d, n in h.copies:
            for m, o in zip(self.model, old):
                m[d, :n] = o[s, :n]
        h.copies = []
        for a, m in zip(self.arrays, self.model):
            assert torch.equal(a, m)


@pytest.mark.parametrize("page", [1, 4, 64])
@pytest.mark.parametrize("deep", [False, True])
def test_fork_shares_full_pages_and_copies_the_rest(page, deep):
    p = Pool([1, page, page + 1, 5 * page - 1 or 1, 0, 0, 0, 0, 0, 0], page=page, n_pages=64, seed=page)
    p.do("fork", [0, 1, 2, 3, 3], [4, 5, 6, 7, 8], deep=deep)
    p.do("fork", [8, 4], [9, -1], deep=not deep)


def test_fork_of_an_empty_sequence_and_of_one_with_missing_pages():
    p = Pool([0, 80, 0, 0, 0], page=16, seed=1)
    p.do("trim", [1], 20, 3)
    p.do("fork", [0, 1, 1], [2, 3, 4], deep=True)


def test_fork_refusals():
    # out of range, a child that is not empty, a child named twice, a parent that is a child, itself
    p = Pool([33, 20, 0, 0, 0, 0, 0, 0], page=16, seed=2)
    p.do("fork", [0, 9, 0, 1, 0, 2, 5, -1], [2, 3, 1, 2, 8, 4, 5, 6])


def test_pages_run_out():
    p = Pool([50, 50, 0, 0, 0], page=16, n_pages=10, seed=3)
    # each deep copy takes 4 of the 2 pages left; a shallow one takes 1
    p.do("fork", [0, 1], [2, 3], deep=True)
    p.do("fork", [0, 1, 0], [2, 3, 4])
    p.do("extend", [0, 1], [60, 64])
    p.do("free", [3])
    p.do("extend", [0, 1], [65, 70])


def test_extend():
    p = Pool([0, 5, 16, 17, 100, 0], page=16, n_pages=64, seed=4)
    p.do("extend", [0, 1, 2, 3, 4], [1, 16, 17, 17, 140])
    p.do("extend", [4, 0, -1, 0, 9, 1], [148, 40, 3, 50, 20, 3])  # twice, out of range, shorter: refused
    p.do("extend", [2], [10 ** 6])  # past the table


def test_free_twice_and_out_of_range():
    p = Pool([30, 40, 50, 0], page=16, seed=5)
    p.do("fork", [0], [3])
    p.do("free", [0, 0, 7, -1])
    p.do("free", [0, 3, 1])
    p.do("free", [0])


def test_counts_that_do_not_add_up_are_recorded():
    p = Pool([30, 30], page=16, seed=6)
    g = p.host.table[0][0]
    p.ref[g] = 0
    p.host.ref[g] = 0
    p.host.table[1][0] = 10 ** 6
    p.table[1, 0] = 10 ** 6
    p.do("free", [0, 1])


@pytest.mark.parametrize("window,n_first", [(1, 0), (17, 0), (16, 1), (33, 40), (1000, 3), (10 ** 15, 10 ** 15)])
def test_trim(window, n_first):
    p = Pool([1, 16, 100, 333, 0], page=16, n_pages=64, seed=7)
    p.do("trim", [3, 0, 2, 3, 4], window, n_first)
    p.do("trim", [1, 3], max(1, window // 2), n_first, [0, 3, 0, 50, 0])
    p.do("free", [3, 1, 2, 0])


@pytest.mark.parametrize("seed", range(4))
def test_compact(seed):
    rng = random.Random(seed)
    p = Pool([rng.randint(0, 200) for _ in range(9)] + [0], page=16, n_pages=150, seed=seed, extra_cols=2)
    p.do("fork", [3], [9]) if p.host.len[3] else None
    p.do("free", [b for b in range(9) if rng.random() < 0.4][:8])
    p.compact()
    p.compact()  # nothing moves


def test_compact_of_an_empty_and_of_a_full_pool():
    p = Pool([0, 0], page=16, n_pages=20, seed=8)
    p.compact()
    p = Pool([160, 160], page=16, n_pages=20, seed=9)
    p.compact()


def test_compact_records_entries_that_name_free_pages():
    p = Pool([16, 16], page=16, n_pages=40, seed=10)
    p.table[0, 1] = 39 if 39 not in (p.host.table[0][0], p.host.table[1][0]) else 38
    p.host.table[0][1] = int(p.table[0, 1])
    p.compact()


@pytest.mark.parametrize("n_pages", [1, 7, 16384, 16385, 40000])
def test_pools_around_the_scan_rounds(n_pages):
    p = Pool([0] * 5, page=1, n_pages=n_pages, cols=n_pages, seed=11, arrays=((torch.uint8, 16),))
    p.do("extend", [0, 1, 2], [n_pages // 2, n_pages // 3, 1])
    p.do("free", [0])
    p.compact()
    p.do("extend", [4, 3], [min(n_pages, 5), n_pages])


@pytest.mark.parametrize("width", [1, 4, 7, 16, 1024])
def test_array_widths_and_alignments(width):
    # rows of any width; odd ones end inside a 16-byte word, and what lies behind the copied rows stays
    p = Pool([100, 37, 0, 0], page=32, n_pages=30, seed=12, arrays=((torch.uint8, width), (torch.uint8, 3)))
    p.arrays.append(torch.zeros(30 * 32 * width + 1, dtype=torch.uint8, device=DEV)[1:].view(30, 32, width))
    p.arrays[-1].copy_(p.arrays[0])
    p.model.append(p.arrays[-1].clone())
    p.do("fork", [0, 1], [2, 3])
    p.do("free", [0])
    p.compact()


def test_strided_layers_and_no_arrays():
    p = Pool([100, 37, 0, 0], page=32, n_pages=30, seed=13, layers=3, extra_cols=4)
    p.do("fork", [0, 1], [2, 3], deep=True)
    p.do("free", [0])
    p.compact()
    q = Pool([100, 0], page=32, n_pages=30, seed=14, arrays=())
    q.do("fork", [0], [1])
    q.compact()


def test_a_captured_call_follows_the_state():
    p = Pool([40, 40, 0, 0], page=16, n_pages=40, seed=15)
    kids, parents = p.ids([2, 3]), p.ids([0, 1])
    grow = p.ids([45, 48], torch.int64)
    calls = [p.ctx.prepare_pages_free(p.pool, kids), p.ctx.prepare_pages_fork(p.pool, parents, kids, p.arrays, p.ws),
             p.ctx.prepare_pages_extend(p.pool, kids, grow, p.ws)]
    p.do("fork", [0, 1], [2, 3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            for c in calls:
                c.run()
    for par in ([0, 1], [1, 1], [0, 0]):
        parents.copy_(torch.tensor(par, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.host.free([2, 3])
        p.host.fork(par, [2, 3])
        p.host.extend([2, 3], [45, 48])
        p.compare()


def test_random_sequences_of_operations():
    rng = random.Random(16)
    p = Pool([rng.randint(0, 90) for _ in range(12)], page=8, n_pages=120, cols=20, seed=16)
    for step in range(60):
        what = rng.choice(["extend", "fork", "free", "trim", "compact"])
        some = [rng.randint(-1, 12) for _ in range(rng.randint(1, 6))]
        if what == "extend":
            p.do("extend", some, [rng.randint(0, 170) for _ in some])
        elif what == "fork":
            p.do("fork", some, [rng.randint(-1, 12) for _ in some], deep=rng.random() < 0.4)
        elif what == "trim":
            p.do("trim", some, rng.randint(1, 60), rng.randint(0, 20))
        elif what == "free":
            p.do("free", some[:2])
        else:
            p.compact()


def test_no_entries_enqueue_nothing():
    p = Pool([40, 0], page=16, seed=17)
    p.do("fork", [], [])
    assert p.ctx.last_launch_count == 0
    p.do("extend", [], [])
    p.do("free", [])


def test_refusals():
    from compressed_sparse_attention_gb300 import binding
    p = Pool([40, 0], page=16, seed=18)
    lib, h, C = p.ctx.lib, p.ctx.h, binding.C
    ids = p.ids([0])
    before = p.table.clone()

    def free(**kw):
        a = binding.PagePoolArgs.from_buffer_copy(p.pool.args)
        n = kw.pop("n", 1)
        seqs = kw.pop("seqs", ids.data_ptr())
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.csa2_pages_free(h, None, C.byref(a), n, seqs)

    assert free(page_size=3) == 2 and free(page_size=1 << 13) == 2
    for kw in (dict(n=-1), dict(n=3), dict(seqs=None), dict(n_pages=0), dict(n_seq=0), dict(table=None), dict(seq_len=None),
               dict(ref=None), dict(table_ld=1), dict(max_pages=0)):
        assert free(**kw) == 1, kw
    assert lib.csa2_pages_free(h, None, None, 1, ids.data_ptr()) == 1
    for window, n_first in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(binding.Csa2Error):
            p.ctx.pages_trim(p.pool, ids, window, n_first)
    size = p.ws.numel()
    ext = lambda ws, n: lib.csa2_pages_extend(h, None, C.byref(p.pool.args), 1, ids.data_ptr(),  # noqa: E731
                                              p.seq_len.data_ptr(), ws, n)
    assert ext(None, size) == 6 and ext(p.ws.data_ptr(), size - 1) == 6 and ext(p.ws.data_ptr() + 8, size) == 1
    arr = (binding.PageArray * 1)()
    arr[0].base, arr[0].page_stride, arr[0].row_bytes = p.arrays[0].data_ptr(), 16 * 16, 16
    fork = lambda n: lib.csa2_pages_fork(h, None, C.byref(p.pool.args), 1, ids.data_ptr(), ids.data_ptr(), 0, n,  # noqa: E731
                                         arr, p.ws.data_ptr(), size)
    assert fork(129) == 2 and fork(-1) == 1
    arr[0].page_stride = 255
    assert fork(1) == 1
    arr[0].page_stride, arr[0].row_bytes = 256, 0
    assert fork(1) == 1
    with pytest.raises(ValueError):
        p.ctx.pages_fork(p.pool, ids, ids, [p.arrays[0][:, :8]], p.ws)
    torch.cuda.synchronize()
    assert torch.equal(p.table, before) and p.ctx.check()[0] == 0


def test_more_sequences_than_the_plan_holds_in_shared_memory():
    n = 2500
    p = Pool([3] * 6 + [0] * (n - 6), page=4, n_pages=6000, cols=3, seed=19, arrays=((torch.uint8, 16),))
    p.do("extend", list(range(n)), [5 if b % 2 else 3 for b in range(n)])
    p.do("free", list(range(6, n, 3)))
    p.do("fork", [1, 1, 5], [6, 9, 12])
    p.do("fork", [0, 4, 4], [15, 18, 21], deep=True)
    p.compact()


def test_trim_where_the_first_position_lies_past_every_row():
    p = Pool([40, 33, 8], page=8, seed=20)
    p.do("trim", [0, 1, 2], 16, 10 ** 15, [2 ** 62 + 5, 20, -3])


def test_refuses_misaligned_elements():
    from compressed_sparse_attention_gb300 import binding
    p = Pool([40, 0], page=16, seed=21)
    lib, h, a = p.ctx.lib, p.ctx.h, binding.C.byref(p.pool.args)
    ids, lens, ws, size = p.ids([0, 1]).data_ptr(), p.seq_len.data_ptr(), p.ws.data_ptr(), p.ws.numel()
    before = p.table.clone()
    assert lib.csa2_pages_extend(h, None, a, 1, ids + 2, lens, ws, size) == 1
    assert lib.csa2_pages_extend(h, None, a, 1, ids, lens + 4, ws, size) == 1
    assert lib.csa2_pages_fork(h, None, a, 1, ids + 2, ids, 0, 0, None, ws, size) == 1
    assert lib.csa2_pages_fork(h, None, a, 1, ids, ids + 1, 0, 0, None, ws, size) == 1
    assert lib.csa2_pages_free(h, None, a, 1, ids + 2) == 1
    assert lib.csa2_pages_trim(h, None, a, 1, ids, 4, 0, lens + 4) == 1
    assert lib.csa2_pages_compact(h, None, a, 0, None, ids + 2, ws, size) == 1
    torch.cuda.synchronize()
    assert torch.equal(p.table, before) and p.ctx.check()[0] == 0


@pytest.mark.parametrize("field", ["n_pages", "n_seq"])
def test_refuses_more_pages_or_sequences_than_the_plans_count(field):
    # in the last thousands below 2^31 a plan's 32-bit counters pass the end; refused before anything is read
    from compressed_sparse_attention_gb300 import binding
    p = Pool([40, 0], page=16, seed=22, arrays=((torch.bfloat16, 512),))
    lib, h, C = p.ctx.lib, p.ctx.h, binding.C
    ids, lens, ws, size = p.ids([0, 1]).data_ptr(), p.seq_len.data_ptr(), p.ws.data_ptr(), p.ws.numel()
    before = p.table.clone(), p.ref.clone(), p.seq_len.clone()
    a = binding.PagePoolArgs.from_buffer_copy(p.pool.args)
    pages = torch.zeros((64, 16, 512), dtype=torch.bfloat16, device=DEV)
    kv = binding.PagedKVArgs.from_buffer_copy(p.ctx.paged_kv(pages, p.table).args)
    q = torch.zeros((2, 64, 512), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3.0)
    aws = binding.workspace(p.ctx.attend_paged_workspace_size(1), DEV)
    for n in (2 ** 30 + 1, 2 ** 31 - 4096, 2 ** 31 - 1):
        setattr(a, field, n)
        setattr(kv, field, n)
        assert lib.csa2_pages_extend(h, None, C.byref(a), 1, ids, lens, ws, size) == 2
        assert lib.csa2_pages_fork(h, None, C.byref(a), 1, ids, ids + 4, 0, 0, None, ws, size) == 2
        assert lib.csa2_pages_free(h, None, C.byref(a), 1, ids) == 2
        assert lib.csa2_pages_trim(h, None, C.byref(a), 1, ids, 4, 0, None) == 2
        assert lib.csa2_pages_compact(h, None, C.byref(a), 0, None, None, ws, size) == 2
        assert lib.csa2_attend_paged(h, None, C.byref(kv), 1, q.data_ptr(), lens, ids, None, 0, 0, None, out.data_ptr(),
                                     None, aws.data_ptr(), aws.numel()) == 2
        assert lib.csa2_append_paged(h, None, C.byref(kv), 0, q.data_ptr(), 1, lens, lens) == 2
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, (p.table, p.ref, p.seq_len)))
    assert (out == 3).all() and p.ctx.last_launch_count == 0 and p.ctx.check()[0] == 0


@pytest.mark.parametrize("n_pages", [2047, 2048, 2049, 4095, 4096, 4097, 8191, 8192, 8193])
def test_pools_around_the_plans_rounds(n_pages):
    # fresh pages are looked for 2,048 counts a round, 8,192 in pools above that size; compaction goes by 4,096
    p = Pool([0] * 6, page=1, n_pages=n_pages, cols=n_pages, seed=23, arrays=((torch.uint8, 16),))
    p.do("extend", [0, 1, 2], [n_pages // 2, n_pages // 3, 1])
    p.do("free", [0])
    p.compact()
    p.do("fork", [1, 2], [5, 0], deep=True)
    p.do("free", [1])
    p.do("extend", [4, 3], [min(n_pages, 5), n_pages])  # the second: not enough pages
    p.do("extend", [3], [p.host.ref.count(0)])          # exactly all that are left
    p.do("free", [4, 5])
    p.compact()


@pytest.mark.parametrize("n", [2047, 2048, 2049])
def test_sequences_around_what_the_plan_holds_in_shared_memory(n):
    p = Pool([3] * 6 + [0] * (n - 6), page=4, n_pages=6000, cols=3, seed=24, arrays=((torch.uint8, 16),))
    p.do("extend", list(range(n - 1, -1, -1)), [5 if b % 2 else 3 for b in range(n)])
    p.do("free", list(range(6, n, 3)) + [n - 1])
    p.do("fork", [1, 1, 5], [6, 9, n - 1])
    p.do("fork", [0, 4, 4], [15, 18, 21], deep=True)
    p.compact()


def test_copies_past_32_bits():
    # pages of 128 KB: the source past 8 GB, the copies from the pool's start and back again
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    n_pages, page, width = 70000, 64, 2048
    a = torch.empty((n_pages, page, width), dtype=torch.uint8, device=DEV)
    a[-2:] = torch.randint(0, 256, (2, page, width), generator=torch.Generator().manual_seed(25), dtype=torch.uint8).to(DEV)
    a[:3] = 7
    want = a[-2:].clone()
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    table[0, :2] = torch.tensor([n_pages - 1, n_pages - 2], dtype=torch.int32)
    ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    ref[-2:] = 1
    seq_len = torch.tensor([page + 9, 0], dtype=torch.int64, device=DEV)
    pool = ctx.page_pool(table, seq_len, ref, page)
    ws = binding.workspace(ctx.pages_workspace_size(pool), DEV)
    ids = Pool.ids
    ctx.pages_fork(pool, ids([0]), ids([1]), [a], ws, deep=True)
    assert ctx.check()[0] == 0 and table[1].tolist() == [0, 1, -1]
    assert torch.equal(a[0], want[1]) and torch.equal(a[1, :9], want[0, :9]) and (a[1, 9:] == 7).all()
    n_live = ids([0])
    ctx.pages_compact(pool, [a], n_live, ws)
    assert ctx.check()[0] == 0 and n_live.item() == 4 and table.tolist() == [[3, 2, -1], [0, 1, -1]]
    assert torch.equal(a[2:4], want) and ref.sum().item() == 4


def test_a_table_row_of_the_largest_length():
    # 2^30 rows of 4,096 a page
    page, cols = 4096, 2 ** 30 // 4096
    p = Pool([0, 0, 0], page=page, n_pages=cols + 40, cols=cols, seed=26, arrays=())
    p.do("extend", [0, 1], [2 ** 30 - 5000, 17])
    p.do("extend", [0, 1], [2 ** 30, 2 ** 30 + 1])  # the second: past the table
    p.do("fork", [0], [2])
    p.do("free", [0])
    p.do("extend", [1], [4097])
    p.compact()
