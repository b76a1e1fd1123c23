"""Plain 64-bit forms of the paged-cache operators, and the error bounds the
GPU tests hold the kernels to. Everything here is elementary torch in float64
(or integers), written from the entry points' definitions."""
from __future__ import annotations

import math

import torch

from gpu_common import FMT_BF16, code_bytes, geometry, inv_freq, stored_values

HEADS, DIM = 64, 512
U16 = 2.0 ** -8    # bf16: half a step relative to the value
U32 = 2.0 ** -24   # fp32
FMT_NAMES = {"bf16": 0, "fp8": 1, "fp4": 2}
SCALE_WIDTH = {0: 0, 1: 16, 2: 32}


def random_pages(fmt, n_pages, page, seed, device, lead=()):
    """(codes, scales) of random pages: unit-size values in `fmt`."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    shape = (*lead, n_pages, page)
    if fmt == 0:
        return torch.randn((*shape, DIM), generator=g).to(torch.bfloat16).to(device), None
    width = code_bytes(DIM, fmt)
    codes = torch.randint(0, 256, (*shape, width), dtype=torch.uint8, generator=g)
    if fmt == 1:
        codes = torch.where((codes & 127) == 127, codes - 1, codes)  # 0x7f / 0xff are e4m3's NaN
        codes = torch.where((codes & 0x78) > 0x40, codes & 0xC7, codes)  # magnitudes below 4
        scales = torch.randint(125, 128, (*shape, 16), dtype=torch.uint8, generator=g)
    else:
        scales = (0.25 + 0.25 * torch.rand((*shape, 32), generator=g)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.to(device), scales.to(device)


def page_values(codes, scales, fmt):
    """float64 values [n_pages, page, 512] of stored pages."""
    flat = lambda t: None if t is None else t.cpu().reshape(-1, t.shape[-1])  # noqa: E731
    v = stored_values(flat(codes), flat(scales), fmt)
    return torch.from_numpy(v).reshape(*codes.shape[:2], DIM)


def turned(x, angle, half=False, amplitude=1.0):
    """Pairs of x's last axis turned by `angle` [..., pairs], float64."""
    c, s = torch.cos(angle) * amplitude, torch.sin(angle) * amplitude
    if half:
        u, v = x.chunk(2, -1)
        return torch.cat((u * c - v * s, u * s + v * c), -1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2)


def layer_turned(x, pos, cfg):
    """The context's RoPE on the last rope_dim channels, float64."""
    f = torch.from_numpy(inv_freq(geometry(cfg)))
    if f.numel() == 0:
        return x
    r = 2 * f.numel()
    return torch.cat((x[..., :-r], turned(x[..., -r:], torch.as_tensor(pos, dtype=torch.float64) * f)), -1)


def visible(t, lo, window, n_first):
    """Positions a query at t sees, ascending."""
    lo = max(lo, 0)
    return [p for p in range(lo, t + 1) if window == 0 or p > t - window or p < lo + n_first]


def attend_one(values, table_row, page, q, t, lo, window, n_first, sink, cfg):
    """One query's exact output, lse, and the bounds on the kernel's error.

    With w_p the exact weights p_p / den, v_p the rows, o the output:
      * the products take the weights rounded to bf16, the denominator does
        not: |do| <= U16 B, B = sum_p w_p |v_p|;
      * fp32 accumulation over the rows, one rounding for every 16 rows and one
        for each of up to 160 partials: (n / 16 + 160) U32 B;
      * scores: q~ enters as bf16 hi + lo on the rope channels (U16^2 of each
        rotated value left out, and the rotation itself to 4 U32) and sums in
        fp32 over 36 steps: each weight is off by a factor within
        delta_p = tau sum_i |q~_i||v_pi| (40 U32) + tau sum_rope |q~_i||v_pi|
        (U16^2 + 4 U32) + 2^-21 (exp2 and its scaling), so o by at most
        sum_p w_p delta_p |v_p - o| (numerator and denominator alike);
      * the output rounded to bf16: U16 |o|.
    lse moves by at most max_p delta_p, plus 4 U32 of itself and of the
    reference. Channels of a pair share their bounds (the rotation back)."""
    pos = [p for p in visible(t, lo, window, n_first) if p // page < len(table_row) and 0 <= table_row[p // page] < values.shape[0]]
    tau = float(cfg.softmax_scale)
    n = len(pos)
    s0 = torch.full((HEADS,), -math.inf, dtype=torch.float64) if sink is None else sink.double().cpu()
    if n == 0:
        z = torch.zeros((HEADS, DIM), dtype=torch.float64)
        return z, s0, z + 1e-30, torch.full((HEADS,), 1e-6, dtype=torch.float64) + 4 * U32 * torch.nan_to_num(s0.abs(), posinf=0.0)
    rows = torch.stack([values[table_row[p // page], p % page] for p in pos])
    q = layer_turned(q.double().cpu(), t, cfg)
    z = q @ rows.T * tau
    lse = torch.logsumexp(torch.cat((z, s0[:, None]), -1), -1)
    w = torch.exp(z - lse[:, None])
    o = w @ rows
    r = int(cfg.rope_dim)
    mag = tau * (q.abs() @ rows.abs().T)
    rope = tau * (q[:, DIM - r:].abs() @ rows[:, DIM - r:].abs().T) if r else torch.zeros_like(mag)
    delta = 40 * U32 * mag + (U16 ** 2 + 4 * U32) * rope + 2.0 ** -21
    B = w @ rows.abs()
    S = torch.einsum("hn,hnd->hd", w * delta, (rows[None] - o[:, None]).abs())
    bound = (U16 + (n / 16 + 160) * U32) * B + S
    if r:
        both = bound[:, DIM - r:].reshape(HEADS, -1, 2).sum(-1, keepdim=True).expand(-1, -1, 2).reshape(HEADS, r)
        bound = torch.cat((bound[:, :DIM - r], both), -1)
    o = layer_turned(o, -float(t), cfg)
    bound = bound + U16 * o.abs() + 1e-30
    return o, lse, bound, delta.amax(-1) + 8 * U32 * (1 + lse.abs())


def check_attend(out, lse, values, table, page, q, q_pos, seq_of_q, lo, window, n_first, sink, cfg, what=""):
    """Every query against attend_one."""
    got, got_lse = out.double().cpu(), None if lse is None else lse.double().cpu()
    for i, (t, b) in enumerate(zip(q_pos, seq_of_q)):
        if b < 0:
            continue
        o, l, bo, bl = attend_one(values, table[b], page, q[i], t, 0 if lo is None else lo[b], window, n_first, sink, cfg)
        err = (got[i] - o).abs()
        assert torch.isfinite(got[i]).all(), f"{what} query {i}: not finite"
        assert (err <= bo).all(), f"{what} query {i} (t {t}): err {err.max():.3e}, {float((err / bo).max()):.2f} of the bound"
        if got_lse is not None:
            fin = torch.isfinite(l)
            assert torch.equal(torch.isfinite(got_lse[i]), fin), f"{what} query {i}: lse"
            e = (got_lse[i][fin] - l[fin]).abs()
            assert (e <= bl[fin]).all(), f"{what} query {i}: lse off by {e.max():.3e}, bound {bl[fin].min():.3e}"


# ---------------------------------------------------------------- page operations on the host

class HostPool:
    """The page operations restated with Python lists: the state and the flags they record."""

    BAD_PAGE, OUT, BAD_SEQ = 0x40, 0x80, 0x100

    def __init__(self, table, seq_len, ref, page):
        self.table = [list(r) for r in table]
        self.len, self.ref, self.page = list(seq_len), list(ref), page
        self.flags = 0
        self.copies = []  # (source page, destination page, rows)

    def pages(self, n):
        return -(-n // self.page)

    def _take(self, needs):
        """Fresh pages of each entry (None: refused), lowest first in the entries' order."""
        free = [g for g, r in enumerate(self.ref) if r == 0]
        at, got = 0, []
        for need in needs:
            if need is None:
                got.append(None)
                continue
            if need > 0 and at + need > len(free):
                self.flags |= self.OUT
                got.append(None)
            else:
                got.append(free[at:at + need])
            at += need
        return got

    def extend(self, seqs, new_len):
        needs = []
        for i, (b, n) in enumerate(zip(seqs, new_len)):
            ok = 0 <= b < len(self.len) and b not in seqs[:i] and self.len[b] <= n <= len(self.table[0]) * self.page
            if not ok and b != -1:
                self.flags |= self.BAD_SEQ
            needs.append(self.pages(n) - self.pages(self.len[b]) if ok else None)
        for b, n, got in zip(seqs, new_len, self._take(needs)):
            if got is None:
                continue
            j = self.pages(self.len[b])
            for k, g in enumerate(got):
                self.table[b][j + k] = g
                self.ref[g] = 1
            self.len[b] = n

    def fork(self, parents, children, deep=False):
        n_seq, n_pages = len(self.len), len(self.ref)
        needs = []
        for i, (p, c) in enumerate(zip(parents, children)):
            ok = 0 <= p < n_seq and 0 <= c < n_seq and c not in children[:i] and p not in children and self.len[c] == 0
            if not ok:
                if c != -1:
                    self.flags |= self.BAD_SEQ
                needs.append(None)
                continue
            np = self.pages(self.len[p])
            has = [0 <= g < n_pages for g in self.table[p][:np]]
            needs.append(sum(has) if deep else int(self.len[p] % self.page != 0 and has[-1]))
        for p, c, got in zip(parents, children, self._take(needs)):
            if got is None:
                continue
            got = list(got)
            np = self.pages(self.len[p])
            for j in range(np):
                g = self.table[p][j]
                if not 0 <= g < n_pages:
                    self.table[c][j] = -1
                elif deep or (j == np - 1 and self.len[p] % self.page):
                    d = got.pop(0)
                    self.copies.append((g, d, min(self.page, self.len[p] - j * self.page)))
                    self.table[c][j] = d
                    self.ref[d] = 1
                else:
                    self.table[c][j] = g
                    self.ref[g] += 1
            self.len[c] = self.len[p]

    def _drop(self, b, j):
        g = self.table[b][j]
        if g < 0:
            return
        self.table[b][j] = -1
        if g >= len(self.ref) or self.ref[g] <= 0:
            self.flags |= self.BAD_PAGE
        else:
            self.ref[g] -= 1

    def free(self, seqs):
        for b in seqs:
            if not 0 <= b < len(self.len):
                self.flags |= self.BAD_SEQ if b != -1 else 0
                continue
            for j in range(len(self.table[b])):
                self._drop(b, j)
            self.len[b] = 0

    def trim(self, seqs, window, n_first, lo=None):
        for b in seqs:
            if not 0 <= b < len(self.len):
                self.flags |= self.BAD_SEQ if b != -1 else 0
                continue
            keep = set()
            n = self.len[b]
            start = max(0, lo[b]) if lo else 0
            for p in range(n):
                if start <= p < start + n_first or p >= max(start, n - window):
                    keep.add(p // self.page)
            for j in range(self.pages(n)):
                if j not in keep:
                    self._drop(b, j)

    def compact(self):
        live = [g for g, r in enumerate(self.ref) if r > 0]
        L = len(live)
        to = dict(zip([g for g in live if g >= L], [g for g in range(L) if self.ref[g] == 0]))
        for s, d in to.items():
            self.copies.append((s, d, self.page))
            self.ref[d], self.ref[s] = self.ref[s], 0
        for row in self.table:
            for j, g in enumerate(row):
                if g >= L:
                    if g not in to:
                        self.flags |= self.BAD_PAGE
                    row[j] = to.get(g, -1)
        return L
