"""What the paged and rotary entry points refuse before any GPU work, the
frequencies of csa2_rope's tables, and the marshalling of strided tensors, on
the CPU."""
import ctypes as C
import math

import pytest
import torch

from compressed_sparse_attention_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def test_null_contexts_and_tables_are_refused(lib):
    kv, pool, tab = binding.PagedKVArgs(), binding.PagePoolArgs(), binding.RopeTable()
    assert lib.csa2_attend_paged(None, None, C.byref(kv), 1, None, None, None, None, 0, 0, None, None, None, None, 0) == 1
    assert lib.csa2_append_paged(None, None, C.byref(kv), 0, None, 1, None, None) == 1
    assert lib.csa2_pages_extend(None, None, C.byref(pool), 1, None, None, None, 0) == 1
    assert lib.csa2_pages_fork(None, None, C.byref(pool), 1, None, None, 0, 0, None, None, 0) == 1
    assert lib.csa2_pages_free(None, None, C.byref(pool), 1, None) == 1
    assert lib.csa2_pages_trim(None, None, C.byref(pool), 1, None, 1, 0, None) == 1
    assert lib.csa2_pages_compact(None, None, C.byref(pool), 0, None, None, None, 0) == 1
    assert lib.csa2_rope(None, None, C.byref(tab), 0, 1, 1, 2, None, 0, 0, None, None, 0, 0, 0) == 1
    assert lib.csa2_attend_paged_workspace_size(None, 4) == 0
    assert lib.csa2_pages_workspace_size(None, C.byref(pool)) == 0


@pytest.mark.parametrize("kw", [dict(rope_dim=3), dict(rope_dim=-2), dict(rope_dim=514), dict(offset=3), dict(offset=-2)])
def test_rope_tables_of_unsupported_shapes(lib, kw):
    with pytest.raises(binding.Csa2Error) as e:
        binding.rope_table(**{"rope_dim": 64, **kw})
    assert e.value.status == 2


@pytest.mark.parametrize("kw", [dict(theta=0.0), dict(theta=-1.0), dict(theta=math.inf), dict(factor=0.5),
                                dict(factor=math.nan), dict(amplitude=math.inf), dict(scaling="yarn", orig_len=0.0),
                                dict(scaling="yarn", theta=1.0), dict(scaling="yarn", beta_fast=-1.0),
                                dict(scaling="yarn", beta_slow=0.0)])
def test_rope_tables_of_bad_numbers(lib, kw):
    with pytest.raises(binding.Csa2Error) as e:
        binding.rope_table(64, **kw)
    assert e.value.status == 1


def test_rope_tables_of_unknown_names(lib):
    with pytest.raises(KeyError):
        binding.rope_table(64, layout="split")
    with pytest.raises(KeyError):
        binding.rope_table(64, scaling="cubic")
    t = binding.RopeTable()
    assert lib.csa2_rope_table_init(C.byref(t), 64, 0, 2, 1e4, 0, 1.0, 1.0, 1.0, 1.0, 1.0) == 1
    assert lib.csa2_rope_table_init(C.byref(t), 64, 0, 0, 1e4, 4, 1.0, 1.0, 1.0, 1.0, 1.0) == 1
    assert lib.csa2_rope_table_init(None, 64, 0, 0, 1e4, 0, 1.0, 1.0, 1.0, 1.0, 1.0) == 1


@pytest.mark.parametrize("r", [0, 2, 64, 512])
def test_rope_table_frequencies(lib, r):
    theta, s = 20000.0, 8.0
    plain = [theta ** (-2.0 * k / r) for k in range(r // 2)]
    assert list(binding.rope_table(r, theta=theta).freq[:r // 2]) == pytest.approx(plain, rel=1e-14)
    # `factor` is read by the scaled forms only
    assert list(binding.rope_table(r, theta=theta, factor=s).freq[:r // 2]) == pytest.approx(plain, rel=1e-14)
    lin = binding.rope_table(r, theta=theta, scaling="linear", factor=s)
    assert list(lin.freq[:r // 2]) == pytest.approx([f / s for f in plain], rel=1e-14)
    if r > 2:
        base = theta * s ** (r / (r - 2.0))
        ntk = binding.rope_table(r, theta=theta, scaling="ntk", factor=s)
        assert list(ntk.freq[:r // 2]) == pytest.approx([base ** (-2.0 * k / r) for k in range(r // 2)], rel=1e-13)
        # the last pair turns 1/factor as fast, the first as before
        assert ntk.freq[0] == 1.0 and ntk.freq[r // 2 - 1] == pytest.approx(plain[-1] / s, rel=1e-12)
        yarn = binding.rope_table(r, theta=theta, scaling="yarn", factor=s, orig_len=4096.0)
        got = list(yarn.freq[:r // 2])
        assert got[0] == 1.0 and got[-1] == pytest.approx(plain[-1] / s, rel=1e-12)
        assert all(f / s * (1 - 1e-12) <= v <= f * (1 + 1e-12) for f, v in zip(plain, got))


def test_yarn_table_equals_the_contexts_ramp(lib):
    from oracle import csa2_oracle as O
    want = O.yarn_inv_freq(64, 160000.0, 16.0, 65536.0, 32.0, 1.0)
    tab = binding.rope_table(64, theta=160000.0, scaling="yarn", factor=16.0)
    assert list(tab.freq[:32]) == pytest.approx(list(want), rel=1e-14)


class _Cpu(binding.Context):
    """A context's marshalling without its C side."""

    def __init__(self, fmt=0):
        self.device, self.h = torch.device("cpu"), None
        self.cfg = binding.default_config(kv_format=fmt)
        self.lib = binding.load_library()


def test_paged_kv_marshals_strided_pages_and_tables(lib):
    c = _Cpu()
    cache = torch.zeros((10, 3, 16, 512), dtype=torch.bfloat16)
    tab = torch.zeros((4, 9), dtype=torch.int32)[:, :7]
    a = c.paged_kv(cache[:, 1], tab).args
    assert a.pages == cache.data_ptr() + 16 * 1024 and a.page_stride == 3 * 16 * 1024
    assert (a.n_pages, a.page_size, a.n_seq, a.max_pages, a.table_ld) == (10, 16, 4, 7, 9)
    a = _Cpu(2).paged_kv(torch.zeros((5, 8, 256), dtype=torch.uint8), tab, torch.zeros((5, 8, 32), dtype=torch.uint8)).args
    assert (a.page_stride, a.scale_stride) == (8 * 256, 8 * 32)


def test_paged_kv_refuses_what_it_cannot_read(lib):
    c, f8 = _Cpu(), _Cpu(1)
    pages, tab = torch.zeros((10, 16, 512), dtype=torch.bfloat16), torch.zeros((4, 7), dtype=torch.int32)
    for bad in (pages.half(), pages[:, :, :256], pages.view(-1, 512), pages.transpose(0, 1), pages[:, ::2],
                pages[:1].expand(10, 16, 512)):
        with pytest.raises(ValueError):
            c.paged_kv(bad, tab)
    for bad in (tab.long(), tab.t(), tab[0], tab[:, ::2], tab[:1].expand(4, 7)):
        with pytest.raises(ValueError):
            c.paged_kv(pages, bad)
    codes = torch.zeros((10, 16, 512), dtype=torch.uint8)
    for bad in (None, torch.zeros((10, 16, 32), dtype=torch.uint8), torch.zeros((10, 16, 16))):
        with pytest.raises(ValueError):
            f8.paged_kv(codes, tab, bad)


def test_page_arrays_are_checked_against_the_pool(lib):
    c = _Cpu()
    pool = c.page_pool(torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int64),
                       torch.zeros(6, dtype=torch.int32), 8)
    good = torch.zeros((6, 8, 5))
    arr = c._page_arrays(pool, [good, torch.zeros((6, 3, 8, 2), dtype=torch.uint8)[:, 2]])
    assert (arr[0].page_stride, arr[0].row_bytes) == (160, 20)
    assert (arr[1].page_stride, arr[1].row_bytes) == (48, 2)
    for bad in (good[:5], good[:, :4], good[:, :, 0], torch.zeros(6)):
        with pytest.raises(ValueError):
            c._page_arrays(pool, [bad])


def test_yarn_tables_of_an_infinite_length(lib):
    # the ramp would begin at infinity and make every frequency a NaN
    with pytest.raises(binding.Csa2Error) as e:
        binding.rope_table(64, scaling="yarn", factor=4.0, orig_len=math.inf)
    assert e.value.status == 1
    assert binding.rope_table(64, scaling="linear", factor=4.0, orig_len=math.inf).freq[0] == 0.25  # not read
    # an infinite beta only puts an end of the ramp at the first pair
    assert all(0 < f <= 1 for f in binding.rope_table(64, scaling="yarn", factor=4.0, beta_fast=math.inf).freq[:32])


def test_blocks_of_another_format_or_device_are_refused(lib):
    # pages of several layers side by side: an fp8 cache's page stride also passes for a bf16 page, whose reads would
    # leave the tensor behind the last one
    bf16, f8 = _Cpu(), _Cpu(1)
    cache = torch.zeros((10, 3, 16, 512), dtype=torch.uint8)
    tab = torch.zeros((2, 3), dtype=torch.int32)
    kv = f8.paged_kv(cache[:, 2], tab, torch.zeros((10, 16, 16), dtype=torch.uint8))
    q = torch.zeros((1, 64, 512), dtype=torch.bfloat16)
    pos, seq = torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    ws, off, first = torch.zeros(8), torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int64)
    f8.prepare_attend_paged(kv, q, pos, seq, q.clone(), ws)
    f8.prepare_append_paged(kv, torch.zeros((1, 512)), off, first)
    pool = bf16.page_pool(tab, first, torch.zeros(10, dtype=torch.int32), 16)
    other = _Cpu(1)
    other.device = torch.device("meta")
    for c in (bf16, other):
        with pytest.raises(ValueError):
            c.prepare_attend_paged(kv, q, pos, seq, q.clone(), ws)
        with pytest.raises(ValueError):
            c.prepare_append_paged(kv, torch.zeros((1, 512)), off, first)
    ids = torch.zeros(1, dtype=torch.int32, device="meta")
    for call in (lambda: other.prepare_pages_free(pool, ids), lambda: other.prepare_pages_trim(pool, ids, 4),
                 lambda: other.prepare_pages_extend(pool, ids, ids.long(), ids),
                 lambda: other.prepare_pages_fork(pool, ids, ids, [], ids),
                 lambda: other.prepare_pages_compact(pool, [], None, ids)):
        with pytest.raises(ValueError):
            call()


def test_entries_are_one_axis(lib):
    # of a [2, 3] tensor of sequences only the first two would be taken
    c = _Cpu()
    pool = c.page_pool(torch.zeros((8, 3), dtype=torch.int32), torch.zeros(8, dtype=torch.int64),
                       torch.zeros(10, dtype=torch.int32), 16)
    ids, ws = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(8)
    one = torch.zeros(2, dtype=torch.int32)
    for call in (lambda v: c.prepare_pages_free(pool, v), lambda v: c.prepare_pages_trim(pool, v, 4),
                 lambda v: c.prepare_pages_extend(pool, v, one.long(), ws),
                 lambda v: c.prepare_pages_fork(pool, v, one, [], ws)):
        call(one)
        with pytest.raises(ValueError):
            call(ids)
        with pytest.raises(ValueError):
            call(torch.zeros((), dtype=torch.int32))
