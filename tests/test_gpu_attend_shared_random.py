"""csa2_attend_shared on random plans, the plan restated place by place: groups of
unlike sizes, heads and orders that are not what they should be, common lengths
of any size, padding, queries past the table, missing pages, every format and
page size. Flags exactly, outputs within attend_one's bounds."""
import random

import pytest
import torch

from gpu_common import context, require_gpu
from paged_common import DIM, FMT_NAMES, HEADS, attend_one, page_values, random_pages

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD_QUERY, BAD_PAGE = 0x20, 0x40


def random_plan(rng, n, n_seq, width, page, n_pages, bad):
    cap = width * page
    holes = rng.random() < 0.3
    page_of = lambda: rng.randrange(n_pages) if not holes or rng.random() < 0.9 else rng.choice([-1, n_pages, -7, 1 << 30])  # noqa: E731
    table = [[page_of() for _ in range(width)] for _ in range(n_seq)]
    seq = [rng.choice([rng.randrange(n_seq)] * 17 + [-1, -1, n_seq if bad else -1]) for _ in range(n)]
    pos = [rng.choice([rng.randrange(cap)] * 17 + [-1, cap + 3 if bad else 0, -2 if bad else 0]) for _ in range(n)]
    perm = rng.sample(range(n), n)
    order = [rng.choice([perm[k]] * 17 + [-1, n if bad else -1]) for k in range(n)]
    head = []
    while len(head) < n:
        head += [len(head)] * min(n - len(head), rng.choice([1, 1, 2, 3, 4, 9, 40]))
    for _ in range(rng.randint(0, 3) if bad else 0):
        head[rng.randrange(n)] = rng.choice([rng.randrange(n), -1, n, -(1 << 31)])
    shared = [rng.choice([0, rng.randint(-3, cap + 9), rng.randint(0, width) * page, 1 << 40]) for _ in range(n)]
    return table, seq, pos, order, head, shared


def plain_plan(table, page, n_pages, seq, pos, order, head, shared):
    """({query: its view of the table, None for a bad one}, flags)."""
    n, n_seq, width = len(seq), len(table), len(table[0])
    views, flags, run = {}, 0, 0
    for k in range(n):
        if k == 0 or head[k] != head[k - 1]:
            run = k
        i = order[k]
        if head[k] != run or i < -1 or i >= n:
            flags |= BAD_QUERY
            continue
        if i == -1 or seq[i] == -1:
            continue
        if not 0 <= seq[i] < n_seq or pos[i] < -1:
            flags |= BAD_QUERY
            views[i] = None
            continue
        first = order[run] if 0 <= order[run] < n else -1
        first = seq[first] if first >= 0 else -1
        cols = min(max(shared[run], 0) // page, width) if 0 <= first < n_seq else 0
        views[i] = (table[first][:cols] if cols else []) + table[seq[i]][cols:]
        seen = min(pos[i] + 1, width * page)
        if pos[i] >= width * page or any(not 0 <= g < n_pages for g in views[i][:-(-seen // page)]):
            flags |= BAD_PAGE
    return views, flags


@pytest.mark.parametrize("seed", range(48))
def test_random_plans(seed):
    require_gpu()
    from compressed_sparse_attention_gb300 import binding
    rng = random.Random(seed)
    fmt, page = ["bf16", "fp8", "bf16", "fp4"][seed % 4], 1 << rng.randint(0, 8)
    ctx = context(kv_format=fmt)
    n, n_seq = rng.choice([1, 2, 3, 5, 8, 13, 20, 40, 77, 96, 97, 130, 300]), rng.randint(1, 12)
    width = -(-int(2 ** rng.uniform(0, 10)) // page) + rng.randint(0, 2)
    n_pages = rng.randint(1, 2 * n_seq * width + 3)
    table, seq, pos, order, head, shared = random_plan(rng, n, n_seq, width, page, n_pages, rng.random() < 0.5)
    codes, scales = random_pages(FMT_NAMES[fmt], n_pages, page, seed, DEV)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((n, HEADS, DIM), generator=g).to(torch.bfloat16).to(DEV)
    sink = torch.randn((HEADS,), generator=g).to(DEV) if rng.random() < 0.7 else None
    i32, i64 = (lambda v, t=t: torch.tensor(v, dtype=t, device=DEV) for t in (torch.int32, torch.int64))
    out = torch.full((n, HEADS, DIM), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, HEADS), 77.0, device=DEV)
    ws = binding.workspace(ctx.attend_shared_workspace_size(n), DEV)
    ctx.attend_shared(ctx.paged_kv(codes, i32(table), scales), q, i64(pos), i32(seq), i32(order), i32(head), i64(shared), out, ws,
                      sink=sink, lse=lse)
    got, _ = ctx.check()
    views, flags = plain_plan(table, page, n_pages, seq, pos, order, head, shared)
    assert got == flags, f"flags {got:#x}, not {flags:#x}"
    rest = [i for i in range(n) if i not in views]
    assert (out[rest] == 77).all() and (lse[rest] == 77).all()
    values = page_values(codes, scales, FMT_NAMES[fmt])
    for i in rng.sample(sorted(views), min(5, len(views))):
        t = -1 if views[i] is None else pos[i]
        o, l, bo, bl = attend_one(values, views[i] or [], page, q[i], t, 0, 0, 0, sink, ctx.cfg)
        err, far = (out[i].double().cpu() - o).abs(), (lse[i].double().cpu() - l).abs()
        fin = torch.isfinite(l)
        assert (err <= bo).all(), f"query {i} (t {t}): {float((err / bo).max()):.2f} of the bound"
        assert torch.equal(torch.isfinite(lse[i]).cpu(), fin) and (far[fin] <= bl[fin]).all(), f"query {i}: lse"
