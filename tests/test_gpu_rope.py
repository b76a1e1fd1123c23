"""csa2_rope and csa2_append_paged against plain 64-bit forms.

csa2_rope's bound: the rotated value is u cos - v sin in fp32 from a (cos, sin)
within 2^-22 of the exact one (a turn in 64-bit fixed point, rounded to fp32:
2^-24 * pi for the argument, one ulp for the function) scaled by the
amplitude: |error| <= (2^-22 + 4 * 2^-24)(|u| + |v|) amplitude, then one
rounding to the type, half a step of the result. Channels that are not
rotated are equal."""
import math

import pytest
import torch

from gpu_common import assert_rows_close_stored, context, require_gpu
from paged_common import DIM, FMT_NAMES, U32, layer_turned, page_values, random_pages, turned

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}  # half a subnormal step


def exact_freq(r, theta, scaling, factor, orig, fast, slow):
    f = []
    if scaling == "ntk" and r > 2:
        theta *= factor ** (r / (r - 2.0))
    for k in range(r // 2):
        v = theta ** (-2.0 * k / r)
        if scaling == "linear":
            v /= factor
        if scaling == "yarn" and factor > 1:
            lo = max(0.0, math.floor(r * math.log(orig / (fast * 2 * math.pi)) / (2 * math.log(theta))))
            hi = min(r - 1.0, math.ceil(r * math.log(orig / (slow * 2 * math.pi)) / (2 * math.log(theta))))
            hi = hi + 0.001 if hi == lo else hi
            w = min(1.0, max(0.0, (k - lo) / (hi - lo)))
            v = v * (1 - w) + v / factor * w
        f.append(v)
    return torch.tensor(f, dtype=torch.float64)


def table(r, **kw):
    from compressed_sparse_attention_gb300 import binding
    return binding.rope_table(r, **kw)


def check_rope(x0, out, pos, r, offset, layout, f, amplitude=1.0, transpose=False, before=None):
    dt = out.dtype
    x = x0.double().cpu()
    got = out.double().cpu()
    p = pos.double().cpu()
    live = pos.cpu() >= 0
    a = p[:, None, None] * f * (-1 if transpose else 1)
    seg = x[..., offset:offset + r]
    want = turned(seg, a, layout == "half", amplitude)
    size = seg.abs()
    if layout == "half":
        both = size[..., :r // 2] + size[..., r // 2:]
        both = torch.cat((both, both), -1)
    else:
        both = (size[..., 0::2] + size[..., 1::2]).repeat_interleave(2, -1)
    tol = both * abs(amplitude) * (2.0 ** -22 + 4 * U32)
    tol = tol + (want.abs() + tol) * HALF_STEP[dt] + TINY[dt]
    err = (got[..., offset:offset + r] - want).abs()[live]
    assert (err <= tol[live]).all(), f"off by {float((err / tol[live]).max()):.2f} of the bound"
    rest = torch.ones(x.shape[-1], dtype=torch.bool)
    rest[offset:offset + r] = False
    assert torch.equal(got[live][..., rest], x[live][..., rest])
    if before is not None and (~live).any():
        assert torch.equal(got[~live], before.double().cpu()[~live])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dim,r,offset", [(1, 1, 2, 2, 0), (3, 5, 64, 64, 0), (7, 2, 80, 20, 60),
                                                       (33, 3, 96, 34, 0), (5, 1, 512, 64, 448), (2, 7, 128, 6, 2),
                                                       (40, 9, 192, 128, 64), (3, 2, 1024, 512, 512), (2, 3, 34, 0, 0)])
def test_layouts_types_and_parts(dtype, layout, tokens, heads, dim, r, offset):
    require_gpu()
    ctx = context()
    g = torch.Generator().manual_seed(dim + r)
    x = torch.randn((tokens, heads, dim), generator=g).to(dtype).to(DEV)
    pos = torch.randint(0, 5000, (tokens,), generator=g).to(DEV)
    out = torch.full_like(x, 9.0)
    ctx.rope(table(r, layout=layout, offset=offset, theta=10000.0), x, pos, out)
    f = exact_freq(r, 10000.0, "none", 1, 1, 1, 1)
    check_rope(x, out, pos, r, offset, layout, f)
    y = x.clone()
    ctx.rope(table(r, layout=layout, offset=offset, theta=10000.0), y, pos)  # in place
    assert torch.equal(y, out)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("r", [2, 64, 128])
def test_scalings_far_positions_and_amplitude(scaling, r):
    require_gpu()
    ctx = context()
    kw = dict(factor=40.0, orig_len=4096.0, beta_fast=32.0, beta_slow=1.0)
    x = torch.randn((64, 2, 128), generator=torch.Generator().manual_seed(1)).to(DEV)
    pos = torch.tensor([0, 1, 4095, 4096, 131071, 2 ** 22 - 1, 2 ** 31 + 5, 2 ** 33] * 8, device=DEV)
    f = exact_freq(r, 500000.0, scaling, 40.0, 4096.0, 32.0, 1.0)
    out = torch.empty_like(x)
    ctx.rope(table(r, theta=500000.0, scaling=scaling, amplitude=1.37, layout="half", **kw), x, pos, out)
    # angles up to 2^33: double precision leaves 2^33 * 2^-52 of a radian (pos * f rounded, and f itself),
    # beyond the 2^-22 of the bound only past 2^30; those rows are compared with that much more
    far = pos.cpu().double() * 2.0 ** -51
    seg, want = x[..., :r].double().cpu(), turned(x[..., :r].double().cpu(), pos.cpu().double()[:, None, None] * f, True, 1.37)
    both = seg[..., :r // 2].abs() + seg[..., r // 2:].abs()
    tol = torch.cat((both, both), -1) * 1.37 * (2.0 ** -22 + 4 * U32 + far[:, None, None]) + want.abs() * U32
    assert ((out[..., :r].double().cpu() - want).abs() <= tol).all()
    assert torch.equal(out[..., r:], x[..., r:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_transpose_is_the_gradient(layout):
    require_gpu()
    ctx = context()
    tab = table(32, layout=layout, offset=16, amplitude=0.8, theta=1000.0)
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn((5, 3, 64), generator=g).to(DEV) for _ in range(2))
    pos = torch.arange(5, device=DEV) * 77
    dx = torch.empty_like(x)
    ctx.rope(tab, dy, pos, dx, transpose=True)
    check_rope(dy, dx, pos, 32, 16, layout, exact_freq(32, 1000.0, "none", 1, 1, 1, 1), 0.8, True)
    # differences of <rope(x), dy> along 20 directions: the operator is linear, so they are exact but for fp32
    y = lambda v: (ctx.rope(tab, v, pos, (o := torch.empty_like(v))), o)[1].double()  # noqa: E731
    for i in range(20):
        d = torch.randn((5, 3, 64), generator=g).to(DEV)
        diff = ((y(x + d) - y(x - d)) * dy.double()).sum() / 2
        want = (dx.double() * d.double()).sum()
        scale = (y(d).abs() * dy.double().abs()).sum() + (x.double().abs() * dy.double().abs()).sum()
        assert abs(diff - want) <= 2.0 ** -20 * scale


def test_strides_views_and_padding():
    require_gpu()
    ctx = context()
    f = exact_freq(32, 10000.0, "none", 1, 1, 1, 1)
    tab = table(32, offset=8, theta=10000.0)
    g = torch.Generator().manual_seed(3)
    pos = torch.tensor([5, -1, 0, 100, -7, 3], device=DEV)
    # queries and keys of one fused projection, heads-major copies, an odd element offset
    for make in (lambda: torch.randn((6, 10, 64), generator=g).to(torch.bfloat16).to(DEV)[:, 2:7],
                 lambda: torch.randn((5, 6, 64), generator=g).to(torch.bfloat16).to(DEV).transpose(0, 1),
                 lambda: torch.randn((6 * 5 * 65 + 1,), generator=g).to(torch.bfloat16).to(DEV)[1:].view(6, 5, 65)[..., :64],
                 lambda: torch.randn((1, 5, 64), generator=g).to(torch.bfloat16).to(DEV).expand(6, 5, 64)):
        x = make()
        out = torch.full((6, 5, 64), 4.0, dtype=torch.bfloat16, device=DEV)
        before = out.clone()
        ctx.rope(tab, x, pos, out)
        check_rope(x, out, pos, 32, 8, "interleaved", f, before=before)
        wide = torch.full((6, 12, 64), 4.0, dtype=torch.bfloat16, device=DEV)
        ctx.rope(tab, x, pos, wide[:, 3:8])
        assert torch.equal(wide[:, 3:8], out) and (wide[:, :3] == 4).all() and (wide[:, 8:] == 4).all()
        if 0 not in x.stride():
            keep = x.clone()
            ctx.rope(tab, x, pos)
            assert torch.equal(x, torch.where((pos >= 0)[:, None, None], out, keep))


def test_nan_and_inf_stay_in_their_pairs():
    require_gpu()
    ctx = context()
    x = torch.randn((2, 1, 64), generator=torch.Generator().manual_seed(4)).to(DEV)
    clean = torch.empty_like(x)
    pos = torch.tensor([3, 4], device=DEV)
    ctx.rope(table(64), x, pos, clean)
    x[0, 0, 10], x[1, 0, 21] = math.nan, math.inf
    out = torch.empty_like(x)
    ctx.rope(table(64), x, pos, out)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 0, 10:12] = True
    hit[1, 0, 20:22] = True
    assert torch.equal(out[~hit], clean[~hit]) and not torch.isfinite(out[hit]).any()


def test_rope_graph_and_stream():
    require_gpu()
    ctx = context()
    x = torch.randn((50, 4, 128), generator=torch.Generator().manual_seed(5)).to(DEV)
    pos = torch.arange(50, device=DEV)
    want, out = torch.empty_like(x), torch.empty_like(x)
    tab = table(128, layout="half")
    ctx.rope(tab, x, pos, want)
    g = torch.cuda.CUDAGraph()
    call = ctx.prepare_rope(tab, x, pos, out)
    with torch.cuda.graph(g):
        call.run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_rope_refusals():
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    tab = table(32)
    x = torch.zeros((4, 3, 64), device=DEV)
    pos = torch.zeros(4, dtype=torch.int64, device=DEV)
    out = torch.full_like(x, 5.0)
    bad = [dict(table=table(128)), dict(table=table(32, offset=34)), dict(out=torch.zeros((4, 1, 64), device=DEV).expand(4, 3, 64)),
           dict(out=x.view(-1)[:12 * 60].view(4, 3, 60)), dict(x=out.view(-1)[:744].as_strided((4, 3, 62), (186, 62, 1)),
                                                            out=out.view(-1)[2:746].as_strided((4, 3, 62), (186, 62, 1))),
           dict(pos=pos[:3]), dict(pos=pos.int()), dict(out=out.double()), dict(out=out.cpu())]
    for kw in bad:
        with pytest.raises((binding.Csa2Error, ValueError, TypeError)):
            ctx.rope(kw.get("table", tab), kw.get("x", x), kw.get("pos", pos), kw.get("out", out))
    lib, C = ctx.lib, binding.C
    call = lambda **k: lib.csa2_rope(ctx.h, None, C.byref(k.get("tab", tab)), k.get("dt", 2), k.get("n", 4), k.get("h", 3),  # noqa: E731
                                     k.get("d", 64), k.get("x", x.data_ptr()), k.get("xs", 192), 64, pos.data_ptr(),
                                     k.get("o", out.data_ptr()), 192, k.get("oh", 64), 0)
    for k, st in ((dict(dt=3), 2), (dict(d=63), 2), (dict(d=2048), 2), (dict(n=-1), 1), (dict(h=-1), 1), (dict(xs=-64), 1),
                  (dict(oh=32), 1), (dict(x=None), 1), (dict(o=None), 1), (dict(x=x.data_ptr() + 2), 1), (dict(h=70000), 2)):
        assert call(**k) == st, k
    broken = binding.RopeTable.from_buffer_copy(tab)
    broken.rope_dim = 4096
    assert call(tab=broken) == 1
    broken.rope_dim, broken.layout = 32, 5
    assert call(tab=broken) == 1
    torch.cuda.synchronize()
    assert (out == 5).all()


def test_angles_of_very_far_positions():
    # against pi to 100 digits. A frequency's turn is rounded to 2^-64: off by
    # 2^-65 turns a position; the turn (at most a half) to fp32 by 2^-24 of itself
    from decimal import Decimal, getcontext
    require_gpu()
    getcontext().prec = 100
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
    r = 64
    tab = table(r, theta=5.0e5)
    pos = [2 ** 20 + 1, 2 ** 31 - 1, 2 ** 33 + 12345, 2 ** 38 + 7, 3 * 2 ** 37 + 11]
    x = torch.zeros((len(pos), 1, r), device=DEV)
    x[..., 0::2] = 1.0  # (1, 0) -> (cos, sin)
    out = torch.empty_like(x)
    for sign in (1, -1):
        context().rope(tab, x, torch.tensor(pos, device=DEV), out, transpose=sign < 0)
        got = out.cpu().double()
        for i, p in enumerate(pos):
            for k in range(r // 2):
                turn = Decimal(p) * Decimal(tab.freq[k]) / (2 * pi)
                a = float((turn - turn.to_integral_value()) * 2 * pi) * sign
                tol = 2 * math.pi * p * 2.0 ** -65 + math.pi * 2.0 ** -24 + 2.0 ** -23
                assert abs(got[i, 0, 2 * k].item() - math.cos(a)) <= tol and \
                    abs(got[i, 0, 2 * k + 1].item() - math.sin(a)) <= tol, (p, k)


def test_rope_refuses_bad_tables_pointers_and_extents():
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    tab = table(32)
    x = torch.full((4, 3, 64), 2.0, device=DEV)
    pos = torch.zeros(5, dtype=torch.int64, device=DEV)

    def call(t=tab, p=pos.data_ptr(), n=4, stride=192):
        return ctx.lib.csa2_rope(ctx.h, None, binding.C.byref(t), 2, n, 3, 64, x.data_ptr(), stride, 64, p, x.data_ptr(), stride,
                                 64, 0)

    for k, v in ((0, math.inf), (15, math.nan), (3, 2.0 ** 32), (3, -2.0 ** 40)):
        broken = binding.RopeTable.from_buffer_copy(tab)
        broken.freq[k] = v
        assert call(broken) == 1, (k, v)
    broken = binding.RopeTable.from_buffer_copy(tab)
    broken.amplitude = math.nan
    assert call(broken) == 1
    assert call(p=pos.data_ptr() + 4) == 1
    assert call(n=2 ** 40, stride=2 ** 30) == 2
    torch.cuda.synchronize()
    assert (x == 2).all() and ctx.last_launch_count == 0


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [1, 16, 256])
def test_append_rotates_and_stores(fmt, dtype, page):
    require_gpu()
    ctx = context(kv_format=fmt)
    f = FMT_NAMES[fmt]
    new, had = [1, 0, 37, 5, 0], [70000, 3, 0, 15, 8]
    cols = -(-70001 // page)
    n_pages = 60 + sum(-(-n // page) + 1 for n in new)
    codes, scales = random_pages(f, n_pages, page, 1, DEV)
    old = codes.clone(), None if scales is None else scales.clone()
    tab = torch.full((5, cols), -1, dtype=torch.int32)
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).tolist()
    for b, (n, h) in enumerate(zip(new, had)):
        for j in range(h // page, -(-(h + n) // page)):
            tab[b, j] = free.pop()
    g = torch.Generator().manual_seed(2)
    rows = (3 * torch.randn((sum(new) + 2, DIM), generator=g)).to(dtype).to(DEV)  # two rows past the last sequence
    off = torch.tensor([0, 1, 1, 38, 43, 43], device=DEV)
    kv = ctx.paged_kv(codes, tab.to(DEV), scales)
    ctx.append_paged(kv, rows, off, torch.tensor(had, device=DEV))
    assert ctx.check()[0] == 0
    written = torch.zeros(codes.shape[:2], dtype=torch.bool)
    at, exact = [], []
    i = 0
    for b, (n, h) in enumerate(zip(new, had)):
        for k in range(n):
            p = h + k
            gpage = int(tab[b, p // page])
            assert not written[gpage, p % page]
            written[gpage, p % page] = True
            at.append((gpage, p % page))
            exact.append(layer_turned(rows[i].double().cpu(), p, ctx.cfg))
            i += 1
    pick = torch.tensor(at)
    sc = None if scales is None else scales.cpu()[pick[:, 0], pick[:, 1]]
    assert_rows_close_stored(codes.cpu()[pick[:, 0], pick[:, 1]], sc, torch.stack(exact).numpy(), f, "append")
    same = codes.cpu().view(torch.uint8).reshape(*codes.shape[:2], -1)[~written]
    assert torch.equal(same, old[0].cpu().view(torch.uint8).reshape(*codes.shape[:2], -1)[~written])
    if scales is not None:
        assert torch.equal(scales.cpu()[~written], old[1].cpu()[~written])


def test_append_equals_store_rows_bit_for_bit():
    # the same rotation and rounding as the packed form's
    require_gpu()
    for fmt in ("bf16", "fp8", "fp4"):
        ctx = context(kv_format=fmt)
        f = FMT_NAMES[fmt]
        rows = torch.randn((40, DIM), generator=torch.Generator().manual_seed(3)).to(DEV)
        pos = torch.arange(1000, 1040, device=DEV)
        codes, scales = random_pages(f, 8, 8, 4, DEV)
        flat = torch.empty((40, codes.shape[2]), dtype=codes.dtype, device=DEV)
        flat_sc = None if scales is None else torch.empty((40, scales.shape[2]), dtype=torch.uint8, device=DEV)
        ctx.store_rows(rows, pos, f, flat, flat_sc)
        tab = torch.full((1, 130), -1, dtype=torch.int32, device=DEV)
        tab[0, 125:130] = torch.tensor([6, 2, 7, 0, 3], dtype=torch.int32)
        ctx.append_paged(ctx.paged_kv(codes, tab, scales), rows, torch.tensor([0, 40], device=DEV),
                         torch.tensor([1000], device=DEV))
        assert ctx.check()[0] == 0
        got = codes[[6, 2, 7, 0, 3]].reshape(40, -1)
        assert torch.equal(got.view(torch.uint8), flat.view(torch.uint8))
        if scales is not None:
            assert torch.equal(scales[[6, 2, 7, 0, 3]].reshape(40, -1), flat_sc)


def test_append_without_a_page_is_recorded_and_skipped():
    require_gpu()
    ctx = context()
    from compressed_sparse_attention_gb300 import binding
    codes, _ = random_pages(0, 4, 8, 5, DEV)
    old = codes.clone()
    tab = torch.tensor([[1, -1, 10 ** 6], [2, 3, -1]], dtype=torch.int32, device=DEV)
    rows = torch.randn((24 + 3 + 2, DIM), generator=torch.Generator().manual_seed(6)).to(DEV)
    kv = ctx.paged_kv(codes, tab)
    # sequence 0: 24 rows over a page, a missing one and one out of range, 3 past the table; sequence 1 from before 0
    ctx.append_paged(kv, rows, torch.tensor([0, 27, 29], device=DEV), torch.tensor([0, -2], device=DEV))
    assert ctx.check()[0] == binding.FLAG_BAD_PAGE
    want = page_values(old, None, 0)
    want[1] = layer_turned(rows[:8].double().cpu(), torch.arange(8)[:, None], ctx.cfg)
    got = page_values(codes, None, 0)
    assert torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])
    assert (got[1] - want[1]).abs().max() <= 2.0 ** -8 * want[1].abs().max()


def test_append_refusals():
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    codes, _ = random_pages(0, 4, 8, 5, DEV)
    tab = torch.tensor([[1, 2]], dtype=torch.int32, device=DEV)
    kv = ctx.paged_kv(codes, tab)
    rows, off, first = torch.zeros((3, DIM), device=DEV), torch.tensor([0, 3], device=DEV), torch.tensor([0], device=DEV)
    with pytest.raises(TypeError):
        ctx.append_paged(kv, rows.half(), off, first)
    with pytest.raises(ValueError):
        ctx.append_paged(kv, rows[:, :256], off, first)
    with pytest.raises(ValueError):
        ctx.append_paged(kv, rows, off[:1], first)
    with pytest.raises(ValueError):
        ctx.paged_kv(codes.float(), tab)
    with pytest.raises(ValueError):
        ctx.paged_kv(codes.transpose(1, 2), tab)
    lib = ctx.lib
    call = lambda dt=2, n=3, p=rows.data_ptr(): lib.csa2_append_paged(  # noqa: E731
        ctx.h, None, binding.C.byref(kv.args), dt, p, n, off.data_ptr(), first.data_ptr())
    assert call(dt=1) == 2 and call(n=-1) == 1 and call(p=None) == 1 and call(p=rows.data_ptr() + 4) == 1
    assert call(n=0) == 0 and ctx.last_launch_count == 0
    assert lib.csa2_append_paged(ctx.h, None, binding.C.byref(kv.args), 2, rows.data_ptr(), 3, off.data_ptr() + 4,
                                 first.data_ptr()) == 1
    assert lib.csa2_append_paged(ctx.h, None, binding.C.byref(kv.args), 2, rows.data_ptr(), 3, off.data_ptr(),
                                 first.data_ptr() + 4) == 1


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dim", [(1, 5, 64), (6, 1, 64), (6, 5, 64), (300, 4, 24)])
def test_rope_between_parts_of_one_buffer(layout, tokens, heads, dim):
    # x and out are parts of one buffer that share no element, though the span of one holds elements of the other
    require_gpu()
    ctx = context()
    tab = table(16, layout=layout, offset=8, theta=10000.0)
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(0, 4000, (tokens,), generator=g).to(DEV)
    make = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    fused, by_head, wide = make(tokens, 3 * heads, dim), make(2 * heads, tokens, dim), make(tokens, heads, 2 * dim)
    parts = [(fused, fused[:, heads:2 * heads], fused[:, 2 * heads:]), (fused, fused[:, 2 * heads:], fused[:, heads:2 * heads]),
             (by_head, by_head[:heads].transpose(0, 1), by_head[heads:].transpose(0, 1)),
             (by_head, by_head[0::2].transpose(0, 1), by_head[1::2].transpose(0, 1)),
             (wide, wide[..., dim:], wide[..., :dim])]
    for buf, x, out in parts:
        before = buf.clone()
        want = torch.empty((tokens, heads, dim), dtype=buf.dtype, device=DEV)
        ctx.rope(tab, x.clone(), pos, want)
        ctx.rope(tab, x, pos, out)
        assert torch.equal(out, want)
        out.copy_(before.as_strided(out.shape, out.stride(), out.storage_offset()))
        assert torch.equal(buf, before)


def test_rope_refuses_parts_that_overlap():
    from compressed_sparse_attention_gb300 import binding
    require_gpu()
    ctx = context()
    tab = table(16)
    pos = torch.arange(6, device=DEV)
    buf = torch.full((8, 12, 64), 2.0, device=DEV)
    flat = buf.view(-1)
    view = lambda at, tok, head: flat[at:].as_strided((4, 3, 32), (tok, head, 1), flat.storage_offset() + at)  # noqa: E731
    x = view(256, 768, 64)
    for at, tok, head in ((256 + 31, 768, 64), (256 - 31, 768, 64), (256 + 128, 768, 64), (256 + 768, 768, 64),
                          (256 + 64 + 2, 768, 64), (256 + 768 * 3 - 64, 768, 64),  # equal strides: an element in common
                          (256 + 32, 768, 128), (256 + 32, 512, 64)):              # others: within the other's span
        with pytest.raises(binding.Csa2Error) as e:
            ctx.rope(tab, x, pos[:4], view(at, tok, head))
        assert e.value.status == 1, (at, tok, head)
    torch.cuda.synchronize()
    assert (buf == 2).all() and ctx.last_launch_count == 0
    for at in (256 + 32, 256 - 32, 256 + 192, 256 + 768 * 3 + 192):
        out = view(at, 768, 64)
        before = buf.clone()
        ctx.rope(tab, x, pos[:4], out)
        want = torch.empty((4, 3, 32), device=DEV)
        ctx.rope(tab, x.clone(), pos[:4], want)
        assert torch.equal(out, want)
        out.fill_(2.0)
        assert torch.equal(buf, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dim,r,offset", [(1024, 512, 512), (1024, 512, 0), (1022, 2, 600), (1024, 0, 0)])
def test_more_units_a_head_than_threads(dtype, layout, dim, r, offset):
    # one element off every wider alignment: one pair (interleaved) or one element of each member (half) a unit
    require_gpu()
    ctx = context()
    g = torch.Generator().manual_seed(dim + r + offset)
    make = lambda: torch.randn((5 * 3 * dim + 1,), generator=g).to(dtype).to(DEV)[1:].view(5, 3, dim)  # noqa: E731
    x, out = make(), make()
    before = out.clone()
    pos = torch.tensor([0, 17, -1, 4000, 123456], device=DEV)
    tab = table(r, layout=layout, offset=offset, theta=10000.0)
    ctx.rope(tab, x, pos, out)
    check_rope(x, out, pos, r, offset, layout, exact_freq(r, 10000.0, "none", 1, 1, 1, 1), before=before)
    keep = x.clone()
    ctx.rope(tab, x, pos)
    assert torch.equal(x, torch.where((pos >= 0)[:, None, None], out, keep))


def test_rope_offsets_past_32_bits():
    # 2^31 and more elements, 4 GB and more: the last tokens against a small call
    require_gpu()
    ctx = context()
    n, heads, dim = 262200, 64, 128
    x = torch.empty((n, heads, dim), dtype=torch.bfloat16, device=DEV)
    x[-40:] = torch.randn((40, heads, dim), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)
    pos = torch.arange(n, device=DEV)
    for layout in ("interleaved", "half"):
        tab = table(96, layout=layout, offset=16)
        small = torch.empty((40, heads, dim), dtype=torch.bfloat16, device=DEV)
        ctx.rope(tab, x[-40:].clone(), pos[-40:].clone(), small)
        out = torch.empty_like(x)
        ctx.rope(tab, x, pos, out)
        assert torch.equal(out[-40:], small)


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_append_past_32_bits(fmt):
    # pages past 4 GB, and the last rows of a table of 2^30
    require_gpu()
    ctx = context(kv_format=fmt)
    f = FMT_NAMES[fmt]
    page, cols = 64, 2 ** 24
    n_pages = 70000 if f == 0 else 270000
    width = 512 if f == 0 else 256
    codes = torch.zeros((n_pages, page, width), dtype=torch.bfloat16 if f == 0 else torch.uint8, device=DEV)
    scales = None if f == 0 else torch.zeros((n_pages, page, 32), dtype=torch.uint8, device=DEV)
    tab = torch.full((1, cols), -1, dtype=torch.int32, device=DEV)
    tab[0, -2:] = torch.tensor([n_pages - 1, n_pages - 3], dtype=torch.int32)
    rows = torch.randn((70, DIM), generator=torch.Generator().manual_seed(9)).to(DEV)
    first = 2 ** 30 - 70
    ctx.append_paged(ctx.paged_kv(codes, tab, scales), rows, torch.tensor([0, 70], device=DEV), torch.tensor([first], device=DEV))
    assert ctx.check()[0] == 0
    exact = torch.stack([layer_turned(rows[i].double().cpu(), first + i, ctx.cfg) for i in range(70)])
    got = torch.cat((codes[n_pages - 1, 58:], codes[n_pages - 3])).cpu()
    sc = None if scales is None else torch.cat((scales[n_pages - 1, 58:], scales[n_pages - 3])).cpu()
    assert_rows_close_stored(got, sc, exact.numpy(), f, "append")
    assert (codes[n_pages - 2] == 0).all() and (codes[n_pages - 1, :58] == 0).all() and (codes[:n_pages - 3:997] == 0).all()
