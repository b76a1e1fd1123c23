"""The paged operators run together as a serving loop runs them: prompts
appended and attended, sequences forked, decoded apart, trimmed, freed, and the
pool compacted in between; every attention output is checked against the rows
that the sequences were given, kept on the host."""
import random

import pytest
import torch

from gpu_common import context, require_gpu
from paged_common import DIM, FMT_NAMES, HEADS, attend_one, page_values

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt,window,n_first", [("bf16", 0, 0), ("fp8", 0, 0), ("fp4", 0, 0), ("bf16", 24, 3)])
def test_serving_loop(fmt, window, n_first):
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context(kv_format=fmt)
    f, page, n_pages, n_seq, cols = FMT_NAMES[fmt], 16, 48, 6, 12
    width = {0: DIM, 1: DIM, 2: DIM // 2}[f]
    codes = torch.zeros((n_pages, page, width), dtype=torch.bfloat16 if f == 0 else torch.uint8, device=DEV)
    scales = None if f == 0 else torch.zeros((n_pages, page, 16 if f == 1 else 32), dtype=torch.uint8, device=DEV)
    table = torch.full((n_seq, cols), -1, dtype=torch.int32, device=DEV)
    seq_len = torch.zeros(n_seq, dtype=torch.int64, device=DEV)
    ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    pool = ctx.page_pool(table, seq_len, ref, page)
    kv = ctx.paged_kv(codes, table, scales)
    arrays = [codes] + ([scales] if scales is not None else [])
    ws = binding.workspace(ctx.pages_workspace_size(pool), DEV)
    aws = binding.workspace(ctx.attend_paged_workspace_size(1), DEV)
    n_live = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(1)
    rng = random.Random(1)
    stored = [[] for _ in range(n_seq)]  # the values of each sequence's rows, as the cache holds them
    sink = torch.randn(HEADS, generator=g).to(DEV)
    ids = lambda v, dt=torch.int32: torch.tensor(v, dtype=dt, device=DEV)  # noqa: E731

    def append(new):
        """new: {sequence: tokens}; pages, rows and one query at every sequence's last position."""
        seqs = sorted(new)
        had = [len(stored[b]) for b in range(n_seq)]
        ctx.pages_extend(pool, ids(seqs), ids([had[b] + new[b] for b in seqs], torch.int64), ws)
        rows = torch.randn((sum(new.values()), DIM), generator=g).to(DEV)
        off = [0]
        for b in range(n_seq):
            off.append(off[-1] + new.get(b, 0))
        ctx.append_paged(kv, rows, ids(off, torch.int64), ids(had, torch.int64))
        q = torch.randn((len(seqs), HEADS, DIM), generator=g).to(torch.bfloat16).to(DEV)
        out, lse = torch.empty_like(q), torch.empty((len(seqs), HEADS), device=DEV)
        pos = [had[b] + new[b] - 1 for b in seqs]
        ctx.attend_paged(kv, q, ids(pos, torch.int64), ids(seqs), out, aws, sink=sink, lse=lse, window=window,
                         n_first=n_first)
        assert ctx.check()[0] == 0
        # the new rows as stored, read back through the table; the old ones as the host remembers them
        values, rows_of = page_values(codes, scales, f), table.tolist()
        for b in seqs:
            for p in range(had[b], had[b] + new[b]):
                stored[b].append(values[rows_of[b][p // page], p % page])
        for i, (b, t) in enumerate(zip(seqs, pos)):
            mine = torch.stack(stored[b])
            pad = torch.cat((mine, torch.zeros((-len(mine) % page, DIM), dtype=torch.float64))).reshape(-1, page, DIM)
            o, l, bo, bl = attend_one(pad, list(range(pad.shape[0])), page, q[i], t, 0, window, n_first, sink, ctx.cfg)
            assert ((out[i].double().cpu() - o).abs() <= bo).all(), f"sequence {b} at {t}"
            assert ((lse[i].double().cpu() - l).abs() <= bl).all()

    append({0: 50, 1: 17, 2: 5})
    for step in range(6):
        append({b: 1 for b in range(n_seq) if stored[b]})
        if step == 0:
            ctx.pages_fork(pool, ids([0, 0, 1]), ids([3, 4, 5]), arrays, ws)
            for p, c in ((0, 3), (0, 4), (1, 5)):
                stored[c] = list(stored[p])
        elif step == 1 and window:
            ctx.pages_trim(pool, ids([0, 3, 4]), window, n_first)
        elif step == 2:
            ctx.pages_free(pool, ids([0, 2]))
            stored[0], stored[2] = [], []
            ctx.pages_compact(pool, arrays, n_live, ws)
            assert n_live.item() == int((ref > 0).sum()) and (ref[n_live.item():] == 0).all()
        elif step == 3:
            ctx.pages_fork(pool, ids([4]), ids([0]), arrays, ws, deep=True)
            stored[0] = list(stored[4])
        elif step == 4:
            append({1: rng.randint(10, 20), 0: 16})
    ctx.pages_free(pool, ids(list(range(n_seq))))
    assert ctx.check()[0] == 0 and (ref == 0).all() and (table == -1).all() and (seq_len == 0).all()


def test_every_operator_from_a_host_thread_without_cuda_calls():
    # a serving loop's worker thread: its first CUDA call is the library's
    import threading
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    g = torch.Generator().manual_seed(5)
    pages = torch.randn((12, 16, 512), generator=g).to(torch.bfloat16).to(DEV)
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    seq_len, ref = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(12, dtype=torch.int32, device=DEV)
    pool, kv = ctx.page_pool(table, seq_len, ref, 16), ctx.paged_kv(pages, table)
    i32, i64 = (lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)), (lambda *v: torch.tensor(v, device=DEV))
    ws = binding.workspace(ctx.pages_workspace_size(pool), DEV)
    rows = torch.randn((40, 512), generator=g).to(DEV)
    x = torch.randn((4, 2, 64), generator=g).to(DEV)
    out, turned = torch.zeros((1, 64, 512), dtype=torch.bfloat16, device=DEV), torch.zeros_like(x)
    q = torch.randn((1, 64, 512), generator=g).to(torch.bfloat16).to(DEV)
    calls = [ctx.prepare_pages_extend(pool, i32(0), i64(40), ws), ctx.prepare_append_paged(kv, rows, i64(0, 40, 40), i64(0, 0)),
             ctx.prepare_pages_fork(pool, i32(0), i32(1), [pages], ws), ctx.prepare_pages_compact(pool, [pages], i32(0), ws),
             ctx.prepare_attend_paged(kv, q, i64(39), i32(1), out, binding.workspace(ctx.attend_paged_workspace_size(1), DEV)),
             ctx.prepare_pages_trim(pool, i32(0), 16), ctx.prepare_pages_free(pool, i32(0, 1)),
             ctx.prepare_rope(binding.rope_table(64), x, i64(1, 2, 3, 4), turned)]

    def all_of_them(each):
        seq_len.zero_(), ref.zero_(), table.fill_(-1), out.zero_(), turned.zero_()
        torch.cuda.synchronize()
        for c in calls:
            each(c)
            torch.cuda.synchronize()
        return out.clone(), turned.clone(), ref.clone(), table.clone()

    bad = []

    def in_a_thread(c):
        def work():
            try:
                c.run()
            except Exception as e:  # noqa: BLE001
                bad.append(e)
        t = threading.Thread(target=work)
        t.start()
        t.join()

    want = all_of_them(lambda c: c.run())
    got = all_of_them(in_a_thread)
    assert not bad, bad
    assert ctx.check()[0] == 0 and want[0].abs().max() > 0 and (want[3] == -1).all()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
