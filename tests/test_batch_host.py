"""What the batch entry points refuse before any GPU work, and the marshalling
of their structs, on the CPU."""
import ctypes as C

import pytest
import torch

from compressed_sparse_attention_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def test_null_contexts_are_refused(lib):
    kv, pool, batch = binding.PagedKVArgs(), binding.PagePoolArgs(), binding.BatchArgs()
    assert lib.csa2_append_slots(None, None, C.byref(kv), 0, None, 1, None, None) == 1
    assert lib.csa2_batch_tables(None, None, C.byref(pool), 1, None, None, C.byref(batch)) == 1
    assert lib.csa2_query_groups(None, None, None, 1, 1, 1, 16, 1, 1, None, None, 1, None, None, None, None) == 1
    assert lib.csa2_attend_shared(None, None, C.byref(kv), 1, None, None, None, None, None, None, None, None, None, None, 0) == 1
    assert lib.csa2_attend_shared_workspace_size(None, 4) == 0


def test_struct_sizes():
    # seven pointers and two 64-bit sizes less one: table, ld, five arrays, max_tokens
    assert C.sizeof(binding.BatchArgs) == 64
    assert [f[0] for f in binding.BatchArgs._fields_] == ["table", "table_ld", "tok_off", "first_pos", "req_of_tok", "tok_pos",
                                                         "tok_slot", "max_tokens"]


class FakeContext(binding.Context):
    """A context whose tensors live on the CPU: marshalling only."""

    def __init__(self, lib, fmt=binding.KV_BF16):
        self.lib, self.cfg, self.device, self.h = lib, binding.default_config(kv_format=fmt), torch.device("cpu"), None


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def i64(*s):
    return torch.zeros(s, dtype=torch.int64)


def test_batch_tables_marshals_a_strided_table(lib):
    ctx = FakeContext(lib)
    pool = ctx.page_pool(i32(5, 7), i64(5), i32(40), 16)
    wide = i32(3, 11)
    outs = (i64(4), i64(3), i32(9), i64(9), i64(9))
    call = ctx.prepare_batch_tables(pool, i32(3), i64(3), wide[:, :7], *outs)
    a = call._keep[3]
    assert (a.table, a.table_ld, a.max_tokens) == (wide.data_ptr(), 11, 9)
    assert (a.tok_off, a.first_pos, a.req_of_tok, a.tok_pos, a.tok_slot) == tuple(t.data_ptr() for t in outs)


@pytest.mark.parametrize("i,bad", [(0, i32(2)), (1, i64(4)), (2, i32(3, 6)), (3, i64(3)), (4, i64(4)), (5, i32(8)), (6, i64(8)),
                                   (7, i64(10))])
def test_batch_tables_shapes(lib, i, bad):
    ctx = FakeContext(lib)
    pool = ctx.page_pool(i32(5, 7), i64(5), i32(40), 16)
    args = [i32(3), i64(3), i32(3, 7), i64(4), i64(3), i32(9), i64(9), i64(9)]
    args[i] = bad
    with pytest.raises(ValueError):
        ctx.prepare_batch_tables(pool, *args)


def test_batch_tables_types(lib):
    ctx = FakeContext(lib)
    pool = ctx.page_pool(i32(5, 7), i64(5), i32(40), 16)
    good = [i32(3), i64(3), i32(3, 7), i64(4), i64(3), i32(9), i64(9), i64(9)]
    for i, t in enumerate(good):
        args = list(good)
        args[i] = t.to(torch.int64 if t.dtype == torch.int32 else torch.int32)
        with pytest.raises((TypeError, ValueError)):
            ctx.prepare_batch_tables(pool, *args)


def test_query_groups_shapes_and_types(lib):
    ctx = FakeContext(lib)
    good = dict(table=i32(4, 6), page_size=16, n_pages=30, q_pos=i64(5), seq_of_q=i32(5), min_shared=32, order=i32(5), head=i32(5),
                shared=i64(5), n_groups=i32(1))
    ctx.prepare_query_groups(**good)
    for k in ("q_pos", "seq_of_q", "order", "head", "shared", "n_groups"):
        for bad in (good[k][:-1], good[k].to(torch.int64 if good[k].dtype == torch.int32 else torch.int32)):
            with pytest.raises((TypeError, ValueError)):
                ctx.prepare_query_groups(**dict(good, **{k: bad}))


def test_caches_without_a_table(lib):
    ctx = FakeContext(lib)
    kv = ctx.paged_kv(torch.zeros((3, 16, 512), dtype=torch.bfloat16))
    assert (kv.args.table, kv.args.n_seq, kv.args.max_pages, kv.args.n_pages, kv.args.page_size) == (None, 0, 0, 3, 16)
    ctx.prepare_append_slots(kv, torch.zeros((2, 512), dtype=torch.bfloat16), None, i64(2))
    for kw in (dict(rows=torch.zeros((2, 511))), dict(rows=torch.zeros((2, 512), dtype=torch.float16)), dict(pos=i64(3)),
               dict(slots=i64(1)), dict(slots=i32(2)), dict(pos=i32(2))):
        a = dict(kv=kv, rows=torch.zeros((2, 512)), pos=i64(2), slots=i64(2))
        with pytest.raises((TypeError, ValueError)):
            ctx.prepare_append_slots(**dict(a, **kw))


def test_attend_shared_shapes_and_formats(lib):
    ctx = FakeContext(lib)
    kv = ctx.paged_kv(torch.zeros((3, 16, 512), dtype=torch.bfloat16), i32(2, 4))
    q = torch.zeros((5, 64, 512), dtype=torch.bfloat16)
    good = dict(kv=kv, q=q, q_pos=i64(5), seq_of_q=i32(5), order=i32(5), head=i32(5), shared=i64(5), out=torch.zeros_like(q),
                workspace=torch.zeros(64, dtype=torch.uint8), sink=torch.zeros(64), lse=torch.zeros((5, 64)))
    ctx.prepare_attend_shared(**good)
    for k in ("q_pos", "seq_of_q", "order", "head", "shared", "out", "sink", "lse"):
        with pytest.raises(ValueError):
            ctx.prepare_attend_shared(**dict(good, **{k: good[k][:-1]}))
        with pytest.raises(TypeError):
            ctx.prepare_attend_shared(**dict(good, **{k: good[k].to(torch.int16)}))
    with pytest.raises(ValueError):
        FakeContext(lib, binding.KV_FP8).prepare_attend_shared(**good)
