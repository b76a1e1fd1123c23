"""The batch operators of the paged cache as measured work: the tables that a
serving step reads, made from the requests' lengths (page table, token
positions, slots); rows stored by slot; queries grouped by the pages that
their sequences share; and attention that reads what a group shares once for
all of its queries.

Every case runs in two forms that take the same state: the plain one
(elementary torch operations, fp32, rounded once) and, where `own` is set,
the library's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

HEADS, DIM, ROPE = 64, 512, 64  # the layer's geometry: 64 heads share one 512-wide row, its last 64 channels rotated
SCALE = 1.0 / math.sqrt(512.0)
THETA, YARN, ORIG, FAST, SLOW = 160000.0, 16.0, 65536.0, 32.0, 1.0  # the layer's RoPE
ROW_BYTES = {"bf16": 1024, "fp8": 512 + 16, "fp4": 256 + 32}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one prompt of 2K sampled four times: the latency of a small decode step
        dict(name="shared_b4_2k", kind="attend", fmt="bf16", page=64, groups=1, seqs=4, per_seq=1, prefix=2048,
             min_tail=1, max_tail=70),
        # an ordinary serving batch under one system prompt of 8K, with conversations of their own
        dict(name="shared_b32_8k", kind="attend", fmt="bf16", page=64, groups=1, seqs=32, per_seq=1, prefix=8192,
             min_tail=60, max_tail=900),
        # many questions about one long document, the largest
        dict(name="shared_b64_32k", kind="attend", fmt="bf16", page=64, groups=1, seqs=64, per_seq=1, prefix=32768,
             min_tail=30, max_tail=500),
        # five documents with an odd number of readers each, fp8 rows
        dict(name="shared_5x7_16k_fp8", kind="attend", fmt="fp8", page=64, groups=5, seqs=7, per_seq=1, prefix=16000,
             min_tail=5, max_tail=300),
        # a draft token beside the sampled one, fp4 rows, small pages
        dict(name="shared_3x6_9k_fp4_two", kind="attend", fmt="fp4", page=32, groups=3, seqs=6, per_seq=2, prefix=9024,
             min_tail=40, max_tail=700),
        # a search's hypotheses: several prompts, each with a few branches; short pages
        dict(name="shared_12x4_3k", kind="attend", fmt="bf16", page=16, groups=12, seqs=4, per_seq=1, prefix=3008,
             min_tail=2, max_tail=190),
        # a decode step's tables: 64 requests, a token each, from a pool of 8K-token sequences
        dict(name="tables_decode_b64", kind="tables", page=64, n_req=64, n_pool=96, min_len=300, max_len=8191,
             prompts=0, min_new=1, max_new=1, spare=0),
        # a mixed step: 512 requests, some of them with chunks of their prompts, from long sequences; a padded batch
        dict(name="tables_mixed_b512", kind="tables", page=64, n_req=512, n_pool=700, min_len=2000, max_len=131072,
             prompts=24, min_new=1, max_new=700, spare=777),
        # which of 64 decoding requests share a document
        dict(name="groups_b64", kind="groups", page=64, groups=5, queries=64, min_len=2000, max_len=16000, shared=1920),
        # the same for a large batch of short shared prompts
        dict(name="groups_b2047", kind="groups", page=16, groups=130, queries=2047, min_len=700, max_len=5000,
             shared=512),
        # a decode step's new rows, one a request
        dict(name="slots_decode_b32", kind="slots", page=64, rows=32, n_pages=600, dtype="bf16", far=100000, padded=0),
        # a prompt's rows in fp32, as an fp32 normalisation leaves them, with the padding of a fixed-size batch
        dict(name="slots_prompt_8191", kind="slots", page=64, rows=8191, n_pages=150, dtype="fp32", far=1000000,
             padded=200),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "attend", "tables", "groups", "slots"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if kind == "attend":
        groups, per = _log(rng, 1, 12), rng.choice([1, 1, 2, 3])
        seqs = _log(rng, 1, max(1, min(64, 96 // (groups * per))))
        # a drawn case scores at most about as many rows as the listed ones
        most = min(32768, 2000000 // (groups * seqs * per))
        tail = _log(rng, max(per, 2), 1000)
        return dict(kind="attend", fmt=rng.choice(["bf16", "bf16", "fp8", "fp4"]), page=page, groups=groups, seqs=seqs,
                    per_seq=per, prefix=_log(rng, 1, max(2, most - tail)), min_tail=max(per, tail // _log(rng, 1, 12)),
                    max_tail=tail)
    if kind == "tables":
        n = _log(rng, 1, 600)
        hi = _log(rng, 64, 131072)
        new = _log(rng, 1, min(hi, 700))
        return dict(kind="tables", page=page, n_req=n, n_pool=n + rng.randint(0, 200), min_len=max(1, new, hi // 50),
                    max_len=max(hi, new), prompts=min(n, rng.choice([0, 1, 24])), min_new=1, max_new=new,
                    spare=rng.choice([0, 0, rng.randint(1, 1000)]))
    if kind == "groups":
        hi = _log(rng, 2 * page, 32768)
        n = _log(rng, 1, min(2047, 600000 * page // hi))
        return dict(kind="groups", page=page, groups=min(n, _log(rng, 1, 300)), queries=n, min_len=max(1, hi // 6),
                    max_len=hi, shared=_log(rng, 1, hi))
    rows = _log(rng, 1, 8191)
    return dict(kind="slots", page=page, rows=rows, n_pages=-(-rows // page) + rng.randint(1, 300),
                dtype=rng.choice(["bf16", "fp32"]), far=_log(rng, 10, 4000000), padded=rng.choice([0, rng.randint(0, rows)]))


def _spread(n, lo, hi):
    """n lengths between lo and hi, the first the largest (the golden ratio's multiples spread the rest)."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _pages(n, page):
    return -(-n // page)


# ---------------------------------------------------------------- inputs

def _quantised(x):
    """Rows [..., 512] fp32 as e4m3 codes and the power-of-two scales of 32 channels each."""
    blocks = x.reshape(*x.shape[:-1], 16, 32)
    exp = torch.ceil(torch.log2(blocks.abs().amax(-1).clamp_min(2.0 ** -100) / 448.0))
    codes = (blocks * torch.exp2(-exp)[..., None]).to(torch.float8_e4m3fn).reshape(x.shape)
    return codes.view(torch.uint8), (exp + 127).to(torch.uint8)


def _rows(shape, fmt, g):
    """Cache rows as a layer leaves them: unit normal, one row in a hundred four times as large."""
    if fmt == "fp4":  # uniform codes under scales that bring them to unit size
        codes = torch.randint(0, 256, (*shape, DIM // 2), dtype=torch.uint8, device=DEV, generator=g)
        scale = 0.25 + 0.25 * torch.rand((*shape, DIM // 16), device=DEV, generator=g)
        return codes, scale.to(torch.float8_e4m3fn).view(torch.uint8)
    x = torch.randn((*shape, DIM), device=DEV, generator=g)
    x *= torch.where(torch.rand((*shape, 1), device=DEV, generator=g) < 0.01, 4.0, 1.0)
    return (x.to(torch.bfloat16), None) if fmt == "bf16" else _quantised(x)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def _prepare_attend(case, s, g, rng):
    """Sequences whose first pages are their group's, as forks of one prompt leave them. The prefix is cut to whole
    pages, which are what sequences share; the rest of it belongs to each sequence itself."""
    page, n_groups, n_seq, per = case["page"], case["groups"], case["seqs"], case["per_seq"]
    whole = case["prefix"] // page
    tails = _spread(n_groups * n_seq, case["min_tail"], case["max_tail"])
    lens = [case["prefix"] + t for t in tails]
    n_pages = n_groups * whole + sum(_pages(n, page) - whole for n in lens) + 3
    free = list(range(n_pages))
    rng.shuffle(free)
    width = max(_pages(n, page) for n in lens)
    table = []
    for i, n in enumerate(lens):
        first = table[-1][:whole] if i % n_seq else [free.pop() for _ in range(whole)]
        row = first + [free.pop() for _ in range(_pages(n, page) - whole)]
        table.append(row + [-1] * (width - len(row)))
    nq = n_groups * n_seq * per
    s["pages"], s["scales"] = _rows((n_pages, page), case["fmt"], g)
    s["table"] = _i32(table)
    s["seq_of_q"] = _i32([b for b in range(len(lens)) for _ in range(per)])
    s["q_pos"] = _i64([n - per + i for n in lens for i in range(per)])
    s["q"] = torch.randn((nq, HEADS, DIM), device=DEV, generator=g).to(torch.bfloat16)
    s["sink"] = torch.randn((HEADS,), device=DEV, generator=g)
    # the batch's plan, kept from step to step: groups of consecutive queries
    size = n_seq * per
    s["order"] = _i32(list(range(nq)))
    s["head"] = _i32([k - k % size for k in range(nq)])
    s["shared"] = _i64([whole * page if k % size == 0 else 0 for k in range(nq)])
    s["whole"], s["tail"] = whole * page, max(lens) - whole * page
    s["out"] = torch.empty((nq, HEADS, DIM), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty((nq, HEADS), device=DEV)


def _prepare_tables(case, s, rng):
    page, n_req, n_pool = case["page"], case["n_req"], case["n_pool"]
    lens = _spread(n_pool, case["min_len"], case["max_len"])
    rng.shuffle(lens)
    width = _pages(case["max_len"], page) + 2
    n_pages = sum(_pages(n, page) for n in lens) + 5
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(rng.randrange(2 ** 31))).to(torch.int32)
    table = torch.full((n_pool, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        k = _pages(n, page)
        table[b, :k] = perm[at:at + k]
        at += k
    s["table"], s["seq_len"] = table.to(DEV), _i64(lens)
    s["ref"] = torch.ones((n_pages,), dtype=torch.int32, device=DEV)
    seqs = rng.sample(range(n_pool), n_req)
    long = set(rng.sample(range(n_req), case["prompts"])) if case["prompts"] else set()
    news = [case["max_new"] if i in long else case["min_new"] for i in range(n_req)]
    s["seqs"], s["n_new"] = _i32(seqs), _i64(news)
    tokens = sum(news) + case["spare"]
    s["batch"] = torch.empty((n_req, width), dtype=torch.int32, device=DEV)
    s["tok_off"] = torch.empty((n_req + 1,), dtype=torch.int64, device=DEV)
    s["first_pos"] = torch.empty((n_req,), dtype=torch.int64, device=DEV)
    s["seq_of_tok"] = torch.empty((tokens,), dtype=torch.int32, device=DEV)
    s["tok_pos"] = torch.empty((tokens,), dtype=torch.int64, device=DEV)
    s["tok_slot"] = torch.empty((tokens,), dtype=torch.int64, device=DEV)


def _group_lengths(case, rng):
    """(document, length) of each query's sequence, the documents of unlike sizes."""
    n, groups = case["queries"], case["groups"]
    docs = [min(int(groups * rng.random() ** 2), groups - 1) for _ in range(n)]
    lens = _spread(n, case["min_len"], case["max_len"])
    rng.shuffle(lens)
    return docs, lens


def _prepare_groups(case, s, rng):
    page, n = case["page"], case["queries"]
    docs, lens = _group_lengths(case, rng)
    # of each document the sequences share a run of pages of their own choice, from the asked length on
    least = max(1, case["shared"] // page)
    pool = iter(range(1 << 30))
    doc_pages = {d: [next(pool) for _ in range(2 * least + 2)] for d in sorted(set(docs))}
    width = _pages(case["max_len"], page) + 1
    table = []
    for d, m in zip(docs, lens):
        k = _pages(m, page)
        share = min(k, rng.choice([least, least + least // 2, 2 * least + 2]))
        row = doc_pages[d][:share] + [next(pool) for _ in range(k - share)]
        table.append(row + [-1] * (width - k))
    s["n_pages"] = next(pool)
    s["table"], s["seq_of_q"], s["q_pos"] = _i32(table), _i32(list(range(n))), _i64([m - 1 for m in lens])
    # the table's cache, of which this operator reads nothing but the table
    s["order"] = torch.empty((n,), dtype=torch.int32, device=DEV)
    s["head"] = torch.empty((n,), dtype=torch.int32, device=DEV)
    s["share"] = torch.empty((n,), dtype=torch.int64, device=DEV)
    s["n_groups"] = torch.empty((1,), dtype=torch.int32, device=DEV)


def _prepare_slots(case, s, g, rng):
    n, page = case["rows"], case["page"]
    s["pages"], _ = _rows((case["n_pages"], page), "bf16", g)
    slots = torch.randperm(case["n_pages"] * page, device=DEV, generator=g)[:n]
    s["pos"] = torch.randint(0, case["far"], (n,), device=DEV, generator=g)
    if case["padded"]:
        slots[n - case["padded"]:] = -1
        s["pos"][n - case["padded"]:] = -1
    s["slots"] = slots
    s["rows_in"] = torch.randn((n, DIM), device=DEV, generator=g).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rng = random.Random(int(seed))
    s = dict(case)
    if case["kind"] == "attend":
        _prepare_attend(case, s, g, rng)
    elif case["kind"] == "tables":
        _prepare_tables(case, s, rng)
    elif case["kind"] == "groups":
        _prepare_groups(case, s, rng)
    else:
        _prepare_slots(case, s, g, rng)
    return s


# ---------------------------------------------------------------- plain forms

def _frequencies():
    """Angles a position of each rotated pair, in 64 bits."""
    i = torch.arange(ROPE // 2, dtype=torch.float64, device=DEV)
    f = THETA ** (-2.0 * i / ROPE)
    edge = lambda turns: ROPE * math.log(ORIG / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
    low, high = max(0.0, math.floor(edge(FAST))), min(ROPE - 1.0, math.ceil(edge(SLOW)))
    ramp = ((i - low) / (high - low)).clamp(0, 1)
    return f * (1 - ramp) + f / YARN * ramp


def _rotated(x, pos, sign):
    """x [..., 512] fp32, its last 64 channels turned by sign * pos * f in adjacent pairs (pos broadcasts over x's
    leading axes)."""
    a = pos.to(torch.float64)[..., None] * _frequencies()
    c, s = torch.cos(a).float(), sign * torch.sin(a).float()
    u, v = x[..., -ROPE::2], x[..., DIM - ROPE + 1::2]
    return torch.cat((x[..., :-ROPE], torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2)), -1)


def _values(codes, scale, fmt):
    """Stored rows as fp32 values."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float().reshape(*codes.shape[:-1], 16, 32)
        return (v * torch.exp2(scale.float() - 127.0)[..., None]).flatten(-2)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat((grid, -grid))
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).reshape(*codes.shape[:-1], 32, 16)
    return (v * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _stored(s, page, at):
    return _values(s["pages"][page, at], None if s["scales"] is None else s["scales"][page, at], s["fmt"])


def _plain_attend(s):
    """Scores and sums over the group's common rows as one product a group, over each query's own rows as a batch of
    products, and one softmax over both."""
    page, whole = s["page"], s["whole"]
    size = s["seqs"] * s["per_seq"]
    seq = s["seq_of_q"].long()
    q = _rotated(s["q"].float(), s["q_pos"][:, None], 1.0)
    p = whole + torch.arange(s["tail"], device=DEV)[None, :]
    seen = p <= s["q_pos"][:, None]
    p = torch.minimum(p, s["q_pos"][:, None])
    own_rows = _stored(s, torch.gather(s["table"][seq].long(), 1, p // page), p % page)
    z_own = (torch.matmul(q, own_rows.transpose(1, 2)) * SCALE).masked_fill(~seen[:, None, :], -math.inf)
    m = torch.maximum(z_own.amax(-1), s["sink"])
    common = []
    for k in range(0, q.shape[0], size):
        pos = torch.arange(whole, device=DEV)
        rows = _stored(s, s["table"][seq[k]].long()[pos // page], pos % page)
        z = torch.matmul(q[k:k + size].reshape(-1, DIM), rows.T).reshape(size, HEADS, whole) * SCALE
        if whole:
            m[k:k + size] = torch.maximum(m[k:k + size], z.amax(-1))
        common.append((z, rows))
    e = torch.exp(z_own - m[..., None])
    den = e.sum(-1) + torch.exp(s["sink"][None, :] - m)
    o = torch.matmul(e, own_rows)
    for i, (z, rows) in enumerate(common):
        at = slice(i * size, (i + 1) * size)
        e = torch.exp(z - m[at][..., None])
        den[at] += e.sum(-1)
        o[at] += torch.matmul(e.reshape(size * HEADS, whole), rows).reshape(size, HEADS, DIM)
    o = _rotated(o / den[..., None], s["q_pos"][:, None], -1.0)
    return o.to(torch.bfloat16), m + torch.log(den)


def _plain_tables(s):
    page = s["page"]
    seq = s["seqs"].long()
    length, row = s["seq_len"][seq], s["table"][seq]
    column = torch.arange(row.shape[1], device=DEV)
    batch = torch.where(column[None, :] < ((length + page - 1) // page)[:, None], row, -1)
    off = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(s["n_new"], 0)))
    first = length - s["n_new"]
    i = torch.arange(s["tok_pos"].shape[0], device=DEV)
    b = torch.searchsorted(off, i, right=True) - 1
    used = b < seq.shape[0]
    c = b.clamp_max(seq.shape[0] - 1)
    pos = torch.where(used, first[c] + i - off[c], -1)
    at = pos.clamp_min(0)
    slot = torch.where(used, batch[c, at // page].long() * page + at % page, -1)
    return batch, off, first, torch.where(used, b, -1).int(), pos, slot


def _plain_groups(s):
    page, table, n = s["page"], s["table"], s["q_pos"].shape[0]
    columns = -(-s["shared"] // page)
    i = torch.arange(n, device=DEV)
    row = table[s["seq_of_q"].long()]
    seen = (s["q_pos"] + 1) // page  # whole pages that a query sees
    key = row[:, columns - 1] if columns <= row.shape[1] else torch.full_like(row[:, 0], -1)
    key = torch.where((seen >= columns) & (key >= 0), key.long(), -1 - i)
    lead = (key[:, None] == key[None, :]).int().argmax(1)  # the lowest query with the same key
    order = torch.argsort(lead, stable=True)
    place = torch.empty_like(order)
    place[order] = i
    head = place[lead[order]]
    alike = (row == row[lead]) & (row >= 0) & (torch.arange(row.shape[1], device=DEV)[None, :] < seen[:, None])
    run = alike.int().cumprod(1).sum(1)
    least = torch.full((n,), 1 << 40, dtype=torch.int64, device=DEV).scatter_reduce(0, lead, run, "amin")
    many = torch.bincount(lead, minlength=n) > 1
    share = torch.where(head == i, torch.where(many, least * page, 0)[order], 0)
    return order.int(), head.int(), share, (head == i).sum().int().reshape(1)


def _plain_slots(s):
    keep = s["slots"] >= 0
    x = _rotated(s["rows_in"].float(), s["pos"], 1.0).to(torch.bfloat16)
    flat = s["pages"].view(-1, DIM)
    flat[s["slots"][keep]] = x[keep]
    return s["pages"]


# ---------------------------------------------------------------- the library's calls

_contexts = {}


def _context(fmt):
    from compressed_sparse_attention_gb300 import binding
    if fmt not in _contexts:
        _contexts[fmt] = binding.Context(kv_format=fmt)
    return _contexts[fmt]


def _own_calls(s):
    """The call of one pass over this state's buffers, prepared once as a serving loop does."""
    from compressed_sparse_attention_gb300 import binding
    ctx = _context(s.get("fmt", "bf16"))
    if s["kind"] == "attend":
        ws = binding.workspace(ctx.attend_shared_workspace_size(s["q"].shape[0]), DEV)
        return ctx.prepare_attend_shared(ctx.paged_kv(s["pages"], s["table"], s["scales"]), s["q"], s["q_pos"],
                                         s["seq_of_q"], s["order"], s["head"], s["shared"], s["out"], ws,
                                         sink=s["sink"], lse=s["lse"])
    if s["kind"] == "tables":
        pool = ctx.page_pool(s["table"], s["seq_len"], s["ref"], s["page"])
        return ctx.prepare_batch_tables(pool, s["seqs"], s["n_new"], s["batch"], s["tok_off"], s["first_pos"],
                                        s["seq_of_tok"], s["tok_pos"], s["tok_slot"])
    if s["kind"] == "groups":
        return ctx.prepare_query_groups(s["table"], s["page"], s["n_pages"], s["q_pos"], s["seq_of_q"], s["shared"],
                                        s["order"], s["head"], s["share"], s["n_groups"])
    return ctx.prepare_append_slots(ctx.paged_kv(s["pages"], None), s["rows_in"], s["pos"], s["slots"])


def _own_run(s):
    call = s.get("call")
    if call is None:
        call = s["call"] = _own_calls(s)
    call.run()
    if s["kind"] == "attend":
        return s["out"], s["lse"]
    if s["kind"] == "tables":
        return s["batch"], s["tok_off"], s["first_pos"], s["seq_of_tok"], s["tok_pos"], s["tok_slot"]
    if s["kind"] == "groups":
        return s["order"], s["head"], s["share"], s["n_groups"]
    return s["pages"]


def run(state):
    if own:
        return _own_run(state)
    return {"attend": _plain_attend, "tables": _plain_tables, "groups": _plain_groups,
            "slots": _plain_slots}[state["kind"]](state)


# ---------------------------------------------------------------- work and 64-bit results

def work(case):
    kind, page = case["kind"], case["page"]
    if kind == "attend":
        whole, per = case["prefix"] // page * page, case["per_seq"]
        lens = [case["prefix"] + t for t in _spread(case["groups"] * case["seqs"], case["min_tail"], case["max_tail"])]
        rows = case["groups"] * whole + sum(n - whole for n in lens)
        seen = sum(n - per + i + 1 for n in lens for i in range(per))
        return {"bytes": rows * ROW_BYTES[case["fmt"]] + len(lens) * per * HEADS * (2 * DIM * 2 + 4),
                "flops": 4.0 * seen * HEADS * DIM}
    if kind == "tables":
        n, width = case["n_req"], _pages(case["max_len"], page) + 2
        new = case["prompts"] * case["max_new"] + (n - case["prompts"]) * case["min_new"]
        used = n * (case["min_len"] + case["max_len"]) / 2 / page  # table entries in use, about
        return {"bytes": 4 * used + 4 * n * width + 36 * n + 20 * (new + case["spare"]), "flops": 0}
    if kind == "groups":
        # of each row the entries up to the first that differs, and the plan
        return {"bytes": case["queries"] * (4 * (case["shared"] / page + 1) + 12 + 16), "flops": 0}
    live = case["rows"] - case["padded"]
    return {"bytes": live * DIM * ((4 if case["dtype"] == "fp32" else 2) + 2) + 16 * case["rows"],
            "flops": 3.0 * live * ROPE}


def _exact_turn(x, pos, sign):
    """The last 64 channels of x [n, ..., 512] as 32 complex numbers, multiplied by e^(i sign pos f)."""
    f = []
    lo = max(0.0, math.floor(ROPE * math.log(ORIG / (FAST * 2 * math.pi)) / (2 * math.log(THETA))))
    hi = min(ROPE - 1.0, math.ceil(ROPE * math.log(ORIG / (SLOW * 2 * math.pi)) / (2 * math.log(THETA))))
    for k in range(ROPE // 2):
        w = min(1.0, max(0.0, (k - lo) / (hi - lo)))
        one = THETA ** (-2.0 * k / ROPE)
        f.append(one * (1 - w) + one / YARN * w)
    ang = sign * pos.double().reshape(-1, *([1] * (x.dim() - 1))) * torch.tensor(f, dtype=torch.float64, device=DEV)
    z = torch.view_as_complex(x[..., -ROPE:].reshape(*x.shape[:-1], ROPE // 2, 2).contiguous())
    z = z * torch.polar(torch.ones_like(ang), ang)
    return torch.cat((x[..., :-ROPE], torch.view_as_real(z).flatten(-2)), -1)


def _exact_values(codes, scale, fmt):
    if fmt == "bf16":
        return codes.double()
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).double() * torch.pow(2.0, scale.double() - 127).repeat_interleave(32, -1)
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV) / 2
    both = torch.empty((*codes.shape[:-1], DIM), dtype=torch.float64, device=DEV)
    both[..., 0::2] = mag[(codes & 7).long()] * (1 - 2 * ((codes >> 3) & 1).double())
    both[..., 1::2] = mag[((codes >> 4) & 7).long()] * (1 - 2 * (codes >> 7).double())
    return both * scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def exact(case, seed):
    if case["kind"] not in ("attend", "slots"):
        return None  # tables and groups are whole numbers
    s = prepare(case, seed)
    if case["kind"] == "slots":
        pages = s["pages"].double()
        x = _exact_turn(s["rows_in"].double(), s["pos"], 1)
        for i, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                pages[at // case["page"], at % case["page"]] = x[i]
        return pages
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    for i, (t, b) in enumerate(zip(s["q_pos"].tolist(), s["seq_of_q"].tolist())):
        # every row that the query sees, through its own sequence's pages
        p = torch.arange(t + 1, device=DEV)
        page, at = s["table"][b].long()[p // case["page"]], p % case["page"]
        rows = _exact_values(s["pages"][page, at], None if s["scales"] is None else s["scales"][page, at], case["fmt"])
        here = torch.tensor([t] * HEADS, device=DEV)
        z = _exact_turn(s["q"][i].double(), here, 1) @ rows.T * SCALE
        lse[i] = torch.logsumexp(torch.cat((z, s["sink"].double()[:, None]), -1), -1)
        out[i] = _exact_turn(torch.exp(z - lse[i][:, None]) @ rows, here, -1)
    return out, lse
