"""csa2_batch_tables, csa2_query_groups and csa2_append_slots at the ends of
their ranges: nothing to do, padded batches, many requests."""
import pytest
import torch

from gpu_common import context, require_gpu
from test_gpu_batch import DEV, i32, i64

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
