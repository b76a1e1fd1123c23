"""The paged-cache operators as measured work: attention of new tokens over a
paged key/value cache (whole, or a sliding window plus the first tokens), the
page operations that grow, share, copy and compact such a cache, rotary
positions, and the append that rotates and stores new rows.

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
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user's short conversation: the latency of a single decode step
        dict(name="decode_b1_2k", kind="attend", fmt="bf16", page=64, n_seq=1, per_seq=1, min_len=2049, max_len=2049,
             window=0, first=0, lo=0),
        # an ordinary serving batch of ragged lengths
        dict(name="decode_b32_ragged_8k", kind="attend", fmt="bf16", page=64, n_seq=32, per_seq=1, min_len=700,
             max_len=8191, window=0, first=0, lo=0),
        # long documents in the fp8 format, the largest dense read
        dict(name="decode_b8_128k_fp8", kind="attend", fmt="fp8", page=64, n_seq=8, per_seq=1, min_len=131072,
             max_len=131072, window=0, first=0, lo=0),
        # fp4 rows, small pages, two tokens a sequence (a draft token beside the sampled one)
        dict(name="decode_b8_20k_fp4_two", kind="attend", fmt="fp4", page=32, n_seq=8, per_seq=2, min_len=9001,
             max_len=20011, window=0, first=0, lo=0),
        # streaming decode: a window of 1,024 and the first 4 tokens, long caches
        dict(name="window_decode_b64", kind="attend", fmt="bf16", page=16, n_seq=64, per_seq=1, min_len=90,
             max_len=32771, window=1024, first=4, lo=0),
        # a prompt chunk under a window: every token of the chunk is a query; left-padded sequences
        dict(name="window_prompt_2x600", kind="attend", fmt="bf16", page=64, n_seq=2, per_seq=600, min_len=2500,
             max_len=2900, window=512, first=4, lo=7),
        # one step of a search over 8 groups of 4 hypotheses: losers freed, winners forked, children grown by a token
        dict(name="pages_search_step", kind="fork", layers=4, page=64, n_pages=2048, groups=8, children=3,
             min_len=900, max_len=2300, deep=False),
        # whole copies of sequences that must not share pages (moved to another user's quota)
        dict(name="pages_copy_deep", kind="fork", layers=4, page=64, n_pages=4096, groups=8, children=1,
             min_len=4001, max_len=8009, deep=True),
        # a pool half of whose pages were freed here and there, moved together
        dict(name="pages_compact", kind="compact", layers=4, page=64, n_pages=4096, n_seq=64, fill=0.5),
        # a decode step's queries, rope part of the head, the layer's own layout
        dict(name="rope_decode_q", kind="rope", n_tok=32, heads=64, head_dim=512, rope=64, offset=448, layout="interleaved",
             scaling="yarn", dtype="bf16", transpose=False, far=100000),
        # a long prompt's queries in the half layout, the whole head rotated; transposed: the gradient's direction
        dict(name="rope_prompt_half", kind="rope", n_tok=8191, heads=64, head_dim=128, rope=128, offset=0, layout="half",
             scaling="linear", dtype="bf16", transpose=True, far=1000000),
        # a prompt's new rows rotated and stored in their pages
        dict(name="append_prompt_16k", kind="append", fmt="bf16", page=64, n_seq=5, min_len=1001, max_len=4096,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "window", "window", "fork", "compact", "rope", "append"])
    if kind in ("attend", "window"):
        n_seq = _log(rng, 1, 64)
        per = rng.choice([1, 1, 2, 3]) if kind == "attend" else rng.choice([1, 2, _log(rng, 2, 300)])
        per = min(per, max(1, 1200 // n_seq))
        # a drawn case reads at most about as many rows as the listed ones
        hi = _log(rng, 1, max(2, min(131072, 500000 // (n_seq * per)))) if kind == "attend" else _log(rng, 1, 32768)
        window = 0 if kind == "attend" else _log(rng, 1, 1200)
        lo = rng.choice([0, 0, rng.randint(1, 40)])
        hi = max(hi, per)
        return dict(kind="attend", fmt=rng.choice(["bf16", "fp8", "fp4"]), page=rng.choice([8, 16, 32, 64, 128, 256]),
                    n_seq=n_seq, per_seq=per, min_len=max(per, hi // _log(rng, 1, 12)), max_len=hi, window=window,
                    first=0 if kind == "attend" else rng.choice([0, 1, 4, rng.randint(2, 200)]), lo=lo)
    if kind == "fork":
        deep = rng.random() < 0.5
        groups, kids = _log(rng, 1, 8), rng.randint(1, 3)
        hi = _log(rng, 1, 4000)
        page = rng.choice([16, 32, 64])
        need = groups * (1 + 2 * kids) * (hi // page + 3)
        return dict(kind="fork", layers=rng.randint(1, 4), page=page, n_pages=need + rng.randint(0, 500), groups=groups,
                    children=kids, min_len=max(1, hi // 3), max_len=hi, deep=deep)
    if kind == "compact":
        n_seq = _log(rng, 1, 64)
        return dict(kind="compact", layers=rng.randint(1, 4), page=rng.choice([16, 32, 64]),
                    n_pages=max(n_seq, _log(rng, 20, 4096)), n_seq=n_seq, fill=rng.uniform(0.05, 0.95))
    if kind == "rope":
        head_dim = rng.choice([32, 64, 80, 96, 128, 192, 256, 512])
        rope = 2 * rng.randint(1, head_dim // 2)
        return dict(kind="rope", n_tok=_log(rng, 1, 8000), heads=_log(rng, 1, 64 * 128 // head_dim), head_dim=head_dim,
                    rope=rope, offset=rng.choice([0, head_dim - rope]), layout=rng.choice(["interleaved", "half"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    transpose=rng.random() < 0.3, far=_log(rng, 10, 4000000))
    hi = _log(rng, 1, 4096)
    return dict(kind="append", fmt="bf16", page=rng.choice([8, 16, 32, 64, 128, 256]), n_seq=_log(rng, 1, 8),
                min_len=max(1, hi // 4), max_len=hi, dtype=rng.choice(["bf16", "fp32"]))


def _lens(n, lo, hi):
    """n lengths between lo and hi, the first the largest (the golden ratio's multiples spread the rest)."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _visible(t, lo, window, first):
    """Number of positions that a query at t sees."""
    if t < lo:
        return 0
    if window == 0:
        return t - lo + 1
    head = min(first, t - lo + 1)
    return head + max(0, t + 1 - max(lo + head, t - window + 1))


# ---------------------------------------------------------------- inputs

def _quantised(x, fmt):
    """Rows [..., 512] fp32 as stored codes and scales."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    if fmt == "fp8":
        blocks = x.reshape(*x.shape[:-1], 16, 32)
        exp = torch.ceil(torch.log2(blocks.abs().amax(-1).clamp_min(2.0 ** -100) / 448.0))
        codes = (blocks * torch.exp2(-exp)[..., None]).to(torch.float8_e4m3fn).reshape(x.shape)
        return codes.view(torch.uint8), (exp + 127).to(torch.uint8)
    raise ValueError(fmt)


def _rows(shape, fmt, g):
    """Cache rows as a layer leaves them: unit normal, one row in a hundred four times as large."""
    if fmt == "fp4":  # uniform codes under scales that bring them to unit size
        codes = torch.randint(0, 256, (*shape, DIM // 2), dtype=torch.uint8, device=DEV, generator=g)
        scale = 0.25 + 0.25 * torch.rand((*shape, DIM // 16), device=DEV, generator=g)
        return codes, scale.to(torch.float8_e4m3fn).view(torch.uint8)
    x = torch.randn((*shape, DIM), device=DEV, generator=g)
    x *= torch.where(torch.rand((*shape, 1), device=DEV, generator=g) < 0.01, 4.0, 1.0)
    return _quantised(x, fmt)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def _table(lens, page, n_pages, rng, width=None):
    """Shuffled pages for sequences of these lengths: (table rows, the pages left over)."""
    free = list(range(n_pages))
    rng.shuffle(free)
    width = width or max(-(-n // page) for n in lens)
    rows = []
    for n in lens:
        k = -(-n // page)
        rows.append([free.pop() for _ in range(k)] + [-1] * (width - k))
    return rows, free


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rng = random.Random(int(seed))
    s = dict(case)
    kind = case["kind"]
    if kind == "attend":
        lens = _lens(case["n_seq"], case["min_len"], case["max_len"])
        n_pages = sum(-(-n // case["page"]) for n in lens) + 3
        s["pages"], s["scales"] = _rows((n_pages, case["page"]), case["fmt"], g)
        s["table"] = _i32(_table(lens, case["page"], n_pages, rng)[0])
        per = case["per_seq"]
        nq = case["n_seq"] * per
        s["seq_of_q"] = _i32([b for b in range(case["n_seq"]) for _ in range(per)])
        s["q_pos"] = _i64([n - per + i for n in lens for i in range(per)])
        s["lo"] = _i64([case["lo"] * (b % 2) for b in range(case["n_seq"])])
        s["q"] = torch.randn((nq, HEADS, DIM), device=DEV, generator=g).to(torch.bfloat16)
        s["sink"] = torch.randn((HEADS,), device=DEV, generator=g)
        # what the caller knows of its batch: the most rows that one query sees
        s["most"] = max(1, max(_visible(n - 1, case["lo"] * (b % 2), case["window"], case["first"])
                               for b, n in enumerate(lens)))
        s["out"] = torch.empty((nq, HEADS, DIM), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((nq, HEADS), device=DEV)
    elif kind == "fork":
        # sequences 0 .. groups-1 live; the others are last step's hypotheses, which hold pages of their own
        kids = case["groups"] * case["children"]
        lens = _lens(case["groups"], case["min_len"], case["max_len"])
        old = [max(1, lens[i % case["groups"]] - 1) for i in range(kids)]
        width = max(lens) // case["page"] + 2
        rows, free = _table(lens + old, case["page"], case["n_pages"], rng, width)
        ref = [1] * case["n_pages"]
        for p in free:
            ref[p] = 0
        s["table"], s["seq_len"], s["ref"] = _i32(rows), _i64(lens + old), _i32(ref)
        s["parents"] = _i32([i % case["groups"] for i in range(kids)])
        s["kids"] = _i32([case["groups"] + i for i in range(kids)])
        s["grown"] = _i64([lens[i % case["groups"]] + 1 for i in range(kids)])
        s["pages"] = torch.randn((case["layers"], case["n_pages"], case["page"], DIM), device=DEV,
                                 generator=g).to(torch.bfloat16)
    elif kind == "compact":
        # sequences of pages that lie anywhere in the pool
        n_live = max(case["n_seq"], int(case["n_pages"] * case["fill"]))
        base, more = divmod(n_live, case["n_seq"])
        lens = [max(1, (base + (i < more)) * case["page"] - i % case["page"]) for i in range(case["n_seq"])]
        rows, free = _table(lens, case["page"], case["n_pages"], rng)
        ref = [1] * case["n_pages"]
        for p in free:
            ref[p] = 0
        s["table0"], s["ref0"], s["seq_len"] = _i32(rows), _i32(ref), _i64(lens)
        s["table"], s["ref"] = s["table0"].clone(), s["ref0"].clone()
        s["n_live"] = _i32([0])
        s["pages"] = torch.randn((case["layers"], case["n_pages"], case["page"], DIM), device=DEV,
                                 generator=g).to(torch.bfloat16)
    elif kind == "rope":
        shape = (case["n_tok"], case["heads"], case["head_dim"])
        s["x"] = torch.randn(shape, device=DEV, generator=g).to(DTYPES[case["dtype"]])
        s["pos"] = torch.randint(0, case["far"], (case["n_tok"],), device=DEV, generator=g)
        s["out"] = torch.empty_like(s["x"])
    else:
        # each sequence already holds some tokens and gets `n` new ones
        new = _lens(case["n_seq"], case["min_len"], case["max_len"])
        had = [(37 * i + 5) % 200 for i in range(case["n_seq"])]
        lens = [a + b for a, b in zip(new, had)]
        n_pages = sum(-(-n // case["page"]) for n in lens) + 2
        s["pages"], s["scales"] = _rows((n_pages, case["page"]), case["fmt"], g)
        s["table"] = _i32(_table(lens, case["page"], n_pages, rng)[0])
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        s["tok_off"], s["first_pos"] = _i64(off), _i64(had)
        s["rows"] = torch.randn((off[-1], DIM), device=DEV, generator=g).to(DTYPES[case["dtype"]])
    return s


# ---------------------------------------------------------------- plain forms

def _frequencies(rope, theta, scaling, factor, orig, fast, slow):
    """Angles a position of each rotated pair, in 64 bits."""
    i = torch.arange(rope // 2, dtype=torch.float64, device=DEV)
    if scaling == "ntk" and rope > 2:
        theta = theta * factor ** (rope / (rope - 2))
    f = theta ** (-2.0 * i / rope)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn" and factor > 1:
        edge = lambda turns: rope * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(0.0, math.floor(edge(fast))), min(rope - 1.0, math.ceil(edge(slow)))
        high = high + 0.001 if high == low else high
        ramp = ((i - low) / (high - low)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp
    return f


def _rotated(x, pos, f, layout, sign):
    """fp32 channels x [..., r] rotated by sign * pos * f (pos broadcasts over x's leading axes)."""
    a = pos.to(torch.float64)[..., None] * f
    c, s = torch.cos(a).float(), sign * torch.sin(a).float()
    if layout == "half":
        u, v = x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
        return torch.cat((u * c - v * s, u * s + v * c), -1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2)


def _layer_rotated(x, pos, sign):
    f = _frequencies(ROPE, THETA, "yarn", YARN, ORIG, FAST, SLOW)
    return torch.cat((x[..., :-ROPE], _rotated(x[..., -ROPE:], pos, f, "interleaved", sign)), -1)


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


def _plain_attend(s):
    seq = s["seq_of_q"].long()
    t, lo = s["q_pos"][:, None], s["lo"][seq][:, None]
    i = torch.arange(s["most"], device=DEV)[None, :]
    if s["window"]:
        head = torch.clamp(torch.minimum(t - lo + 1, torch.full_like(t, s["first"])), min=0)
        p = torch.where(i < head, lo + i, torch.maximum(lo + head, t - s["window"] + 1) + i - head)
    else:
        p = lo + i
    seen = p <= t
    p = torch.minimum(p, t.clamp_min(0))
    page = torch.gather(s["table"][seq].long(), 1, p // s["page"])
    at = p % s["page"]
    rows = _values(s["pages"][page, at], None if s["scales"] is None else s["scales"][page, at], s["fmt"])
    q = _layer_rotated(s["q"].float(), s["q_pos"][:, None], 1.0)
    z = torch.matmul(q, rows.transpose(1, 2)) * SCALE
    z = z.masked_fill(~seen[:, None, :], -math.inf)
    m = torch.maximum(z.amax(-1), s["sink"])[..., None]
    e = torch.exp(z - m)
    den = e.sum(-1, keepdim=True) + torch.exp(s["sink"][None, :, None] - m)
    o = _layer_rotated(torch.matmul(e, rows) / den, s["q_pos"][:, None], -1.0)
    return o.to(torch.bfloat16), (m + torch.log(den))[..., 0]


def _plain_fork(s):
    table, ref, length, page = s["table"], s["ref"], s["seq_len"], s["page"]
    kids, parents = s["kids"].long(), s["parents"].long()
    # free the children's last generation
    held = table[kids]
    ref.index_add_(0, held.clamp_min(0).flatten().long(), -(held >= 0).flatten().int())
    table[kids] = -1
    # fork: shared pages by reference, the partial last page (deep: every page) into the lowest free pages
    row, n = table[parents], length[parents]
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    has = (j < ((n + page - 1) // page)[:, None]) & (row >= 0)
    fresh = has if s["deep"] else has & (j == (n // page)[:, None])
    free = torch.sort(torch.where(ref == 0, torch.arange(ref.numel(), device=DEV), ref.numel()))[0]
    order = (torch.cumsum(fresh.flatten().long(), 0) - 1).clamp_min(0).view_as(fresh)
    child = torch.where(fresh, free[order].int(), torch.where(has, row, -1))
    src, dst = row[fresh].long(), child[fresh].long()
    rows = (n[:, None] - j * page).clamp(0, page)[fresh]
    used = (torch.arange(page, device=DEV)[None, :] < rows[:, None])[None, :, :, None]
    s["pages"][:, dst] = torch.where(used, s["pages"][:, src], s["pages"][:, dst])
    ref.index_add_(0, child.clamp_min(0).flatten().long(), (child >= 0).flatten().int())
    # grow every child by one token: a fresh page where the last one is full
    more = (j >= ((n + page - 1) // page)[:, None]) & (j < ((s["grown"] + page - 1) // page)[:, None])
    free = torch.sort(torch.where(ref == 0, torch.arange(ref.numel(), device=DEV), ref.numel()))[0]
    order = (torch.cumsum(more.flatten().long(), 0) - 1).clamp_min(0).view_as(more)
    new = torch.where(more, free[order].int(), child)
    ref.index_add_(0, new.clamp_min(0).flatten().long(), more.flatten().int())
    table[kids] = new
    length[kids] = s["grown"]
    return s["pages"], table, ref, length


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    ref = s["ref"]
    at = torch.arange(ref.numel(), device=DEV)
    live = ref > 0
    n_live = live.sum()
    src = at[live & (at >= n_live)]
    dst = at[~live & (at < n_live)]
    s["pages"][:, dst] = s["pages"][:, src]
    to = at.clone()
    to[src] = dst
    ref[dst] = ref[src]
    ref[src] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp_min(0).long()].int(), s["table"]))
    s["n_live"].copy_(n_live)
    return s["pages"], s["table"], ref, s["n_live"]


#: factor, original length and ramp of the rope cases' scaled tables
ROPE_CASE = dict(theta=10000.0, factor=8.0, orig=4096.0, fast=32.0, slow=1.0, amplitude=1.1)


def _plain_rope(s):
    k = ROPE_CASE
    f = _frequencies(s["rope"], k["theta"], s["scaling"], k["factor"], k["orig"], k["fast"], k["slow"])
    x = s["x"].float()
    a, b = s["offset"], s["offset"] + s["rope"]
    y = _rotated(x[..., a:b], s["pos"][:, None], f, s["layout"], -1.0 if s["transpose"] else 1.0)
    amp = k["amplitude"] if s["scaling"] == "yarn" else 1.0
    return torch.cat((x[..., :a], y * amp, x[..., b:]), -1).to(s["x"].dtype)


def _plain_append(s):
    i = torch.arange(s["rows"].shape[0], device=DEV)
    b = torch.searchsorted(s["tok_off"], i, right=True) - 1
    p = s["first_pos"][b] + i - s["tok_off"][b]
    x = _layer_rotated(s["rows"].float(), p, 1.0)
    page = s["table"][b, p // s["page"]].long()
    s["pages"][page, p % s["page"]] = x.to(torch.bfloat16)
    return s["pages"]


# ---------------------------------------------------------------- the library's calls

_contexts = {}


def _context(fmt):
    from compressed_sparse_attention_gb300 import binding
    if fmt not in _contexts:
        _contexts[fmt] = binding.Context(kv_format=fmt)
    return _contexts[fmt]


def _own_calls(s):
    """The calls of one pass over this state's buffers, prepared once as a serving loop does."""
    from compressed_sparse_attention_gb300 import binding
    kind = s["kind"]
    ctx = _context(s.get("fmt", "bf16"))
    if kind == "attend":
        ws = binding.workspace(ctx.attend_paged_workspace_size(s["q"].shape[0]), DEV)
        cache = ctx.paged_kv(s["pages"], s["table"], s["scales"])
        return [ctx.prepare_attend_paged(cache, s["q"], s["q_pos"], s["seq_of_q"], s["out"], ws, sink=s["sink"],
                                         lse=s["lse"], lo=s["lo"], window=s["window"], n_first=s["first"])]
    if kind in ("fork", "compact"):
        pool = ctx.page_pool(s["table"], s["seq_len"], s["ref"], s["page"])
        arrays = list(s["pages"].unbind(0))
        ws = binding.workspace(ctx.pages_workspace_size(pool), DEV)
        if kind == "compact":
            return [ctx.prepare_pages_compact(pool, arrays, s["n_live"], ws)]
        return [ctx.prepare_pages_free(pool, s["kids"]),
                ctx.prepare_pages_fork(pool, s["parents"], s["kids"], arrays, ws, deep=s["deep"]),
                ctx.prepare_pages_extend(pool, s["kids"], s["grown"], ws)]
    if kind == "rope":
        k = ROPE_CASE
        tab = binding.rope_table(s["rope"], theta=k["theta"], layout=s["layout"], offset=s["offset"],
                                 scaling=s["scaling"], factor=k["factor"], orig_len=k["orig"], beta_fast=k["fast"],
                                 beta_slow=k["slow"], amplitude=k["amplitude"] if s["scaling"] == "yarn" else 1.0)
        return [ctx.prepare_rope(tab, s["x"], s["pos"], s["out"], transpose=s["transpose"])]
    return [ctx.prepare_append_paged(ctx.paged_kv(s["pages"], s["table"], s["scales"]), s["rows"], s["tok_off"],
                                     s["first_pos"])]


def _own_run(s):
    calls = s.get("calls")
    if calls is None:
        calls = s["calls"] = _own_calls(s)
    kind = s["kind"]
    if kind == "compact":
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
    for c in calls:
        c.run()
    if kind == "attend":
        return s["out"], s["lse"]
    if kind == "fork":
        return s["pages"], s["table"], s["ref"], s["seq_len"]
    if kind == "compact":
        return s["pages"], s["table"], s["ref"], s["n_live"]
    return s["out"] if kind == "rope" else s["pages"]


def run(state):
    if own:
        return _own_run(state)
    return {"attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact, "rope": _plain_rope,
            "append": _plain_append}[state["kind"]](state)


# ---------------------------------------------------------------- work and 64-bit results

def work(case):
    kind = case["kind"]
    if kind == "attend":
        lens, per = _lens(case["n_seq"], case["min_len"], case["max_len"]), case["per_seq"]
        seen = rows = 0
        for b, n in enumerate(lens):
            lo = case["lo"] * (b % 2)
            v = [_visible(t, lo, case["window"], case["first"]) for t in range(n - per, n)]
            seen += sum(v)
            # the distinct rows that the sequence's queries read between them
            if case["window"] == 0:
                rows += max(0, n - lo)
            else:
                t0 = max(lo, n - per - case["window"] + 1)
                rows += max(0, n - t0) + max(0, min(case["first"], t0 - lo, n - lo))
        q = case["n_seq"] * per
        return {"bytes": rows * ROW_BYTES[case["fmt"]] + 2 * q * HEADS * DIM * 2, "flops": 4.0 * seen * HEADS * DIM}
    if kind == "fork":
        lens = _lens(case["groups"], case["min_len"], case["max_len"])
        moved = sum(n if case["deep"] else n % case["page"] for n in lens) * case["children"]
        table = sum(-(-n // case["page"]) for n in lens) * case["children"]
        return {"bytes": 2 * moved * case["layers"] * DIM * 2 + 4 * (4 * table + case["n_pages"]), "flops": 0}
    if kind == "compact":
        n_live = max(case["n_seq"], int(case["n_pages"] * case["fill"]))
        # a live page lies above the n_live-th with the share of pages that are free
        moved = n_live * (1.0 - n_live / case["n_pages"])
        return {"bytes": 2 * moved * case["layers"] * case["page"] * DIM * 2 + 8 * (n_live + case["n_pages"]), "flops": 0}
    if kind == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["n_tok"] * case["heads"] * case["head_dim"]
        return {"bytes": 2 * n * size + 8 * case["n_tok"], "flops": 3.0 * case["n_tok"] * case["heads"] * case["rope"]}
    n = sum(_lens(case["n_seq"], case["min_len"], case["max_len"]))
    return {"bytes": n * (DIM * (4 if case["dtype"] == "fp32" else 2) + ROW_BYTES[case["fmt"]]), "flops": 3.0 * n * ROPE}


def _exact_turn(x, pos, freq, half, sign, amplitude=1.0):
    """Pairs of x's last axis as complex numbers, multiplied by amplitude * e^(i sign pos f)."""
    r = x.shape[-1]
    pairs = torch.complex(x[..., :r // 2], x[..., r // 2:]) if half else torch.view_as_complex(
        x.reshape(*x.shape[:-1], r // 2, 2).contiguous())
    ang = sign * pos.double().reshape(-1, *([1] * (x.dim() - 1))) * freq
    pairs = pairs * torch.polar(torch.full_like(ang, amplitude), ang)
    return torch.cat((pairs.real, pairs.imag), -1) if half else torch.view_as_real(pairs).flatten(-2)


def _exact_freq(r, base, how, factor, orig, fast, slow):
    got = []
    if how == "ntk" and r > 2:
        base *= factor ** (r / (r - 2.0))
    for k in range(r // 2):
        f = base ** (-2.0 * k / r)
        if how == "linear":
            f /= factor
        elif how == "yarn" and factor > 1:
            lo = max(0.0, math.floor(r * math.log(orig / (fast * 2 * math.pi)) / (2 * math.log(base))))
            hi = min(r - 1.0, math.ceil(r * math.log(orig / (slow * 2 * math.pi)) / (2 * math.log(base))))
            w = min(1.0, max(0.0, (k - lo) / ((hi if hi != lo else hi + 0.001) - lo)))
            f = f * (1 - w) + f / factor * w
        got.append(f)
    return torch.tensor(got, dtype=torch.float64, device=DEV)


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
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "attend":
        f = _exact_freq(ROPE, THETA, "yarn", YARN, ORIG, FAST, SLOW)
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
        sink = s["sink"].double()
        pos, seq, cut = s["q_pos"].tolist(), s["seq_of_q"].tolist(), s["lo"].tolist()
        for i, (t, b) in enumerate(zip(pos, seq)):
            p = torch.arange(cut[b], max(cut[b], t + 1), device=DEV)
            if case["window"]:
                p = p[(p > t - case["window"]) | (p < cut[b] + case["first"])]
            page, at = s["table"][b].long()[p // case["page"]], p % case["page"]
            rows = _exact_values(s["pages"][page, at], None if s["scales"] is None else s["scales"][page, at], case["fmt"])
            q = s["q"][i].double()
            here = torch.tensor([t] * HEADS, device=DEV)
            q = torch.cat((q[:, :-ROPE], _exact_turn(q[:, -ROPE:], here, f, False, 1)), -1)
            z = torch.cat((q @ rows.T * SCALE, sink[:, None]), -1)
            lse[i] = torch.logsumexp(z, -1)
            o = torch.exp(z[:, :-1] - lse[i][:, None]) @ rows
            out[i] = torch.cat((o[:, :-ROPE], _exact_turn(o[:, -ROPE:], here, f, False, -1)), -1)
        return out, lse
    if kind == "rope":
        k = ROPE_CASE
        f = _exact_freq(case["rope"], k["theta"], case["scaling"], k["factor"], k["orig"], k["fast"], k["slow"])
        y = s["x"].double()
        at = slice(case["offset"], case["offset"] + case["rope"])
        y[..., at] = _exact_turn(y[..., at].clone(), s["pos"], f, case["layout"] == "half", -1 if case["transpose"] else 1,
                                 k["amplitude"] if case["scaling"] == "yarn" else 1.0)
        return y
    if kind == "append":
        f = _exact_freq(ROPE, THETA, "yarn", YARN, ORIG, FAST, SLOW)
        pages, off, first = s["pages"].double(), s["tok_off"].tolist(), s["first_pos"].tolist()
        for b in range(case["n_seq"]):
            x = s["rows"][off[b]:off[b + 1]].double()
            p = torch.arange(first[b], first[b] + x.shape[0], device=DEV)
            x = torch.cat((x[:, :-ROPE], _exact_turn(x[:, -ROPE:], p, f, False, 1)), -1)
            pages[s["table"][b].long()[p // case["page"]], p % case["page"]] = x
        return pages
    return None  # page operations copy and count: there is nothing to compute
