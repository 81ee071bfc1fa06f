"""Inputs of the 4-bit and gated products for tests that are tighter than a bound on every sum's error (no test
functions here).  Everything is torch on the CPU; `on_gpu` runs a case through the library.

Exact cases: inputs are small whole numbers and powers of two (or scales of 10 bits), chosen so that every partial sum, in
any order, is a multiple of one step below 2^24 of it.  fp32 then rounds nowhere, and an output is the 64-bit result
rounded once: equal, bit for bit.  A gate of 90 and more makes both activations its own value (sigma rounds to 1).

Tight cases: inputs as in use.  The error's root mean square may be 1.01 times that of rounding the 64-bit result to
bf16 once.  That leaves what comes before the rounding 14% of its step's: about 2^-9 / sqrt(3) * 0.14 = 1.6e-4 of a value.
Rounding errors of fp32 sums that are not of one sign make about sqrt(n) * 2^-24 of a partial sum's magnitude, which for
the (24 + q) x of 4-bit weights of one bit (q = -1, 0, 1) is 24 / 0.8 of the sum's own: 1e-4 at n = 2^13 if every sum went
through one chain, and 2e-5 with the group's sums apart, as they are.
"""
from __future__ import annotations

import numpy as np
import torch

from tests.dense_cases import MODS, gen


class Case:
    """x [x_rows, d_in]; W[col][slot] = (weight fp64, q, s) (q and s of 4-bit weights); A, B, scale [col][slot]; ids."""

    def __init__(self, kind, group, ids, slots, d_in, d_out, rank=0, act="silu", fan=1):
        self.kind, self.group, self.ids, self.slots = kind, group, np.asarray(ids, np.int32), slots
        self.d_in, self.d_out, self.rank, self.act, self.fan = d_in, d_out, rank, act, fan
        self.rows = len(self.ids)
        self.is_gated, self.adapted = "gated" in kind, not kind.startswith("grouped")
        self.cols = ("gate", "up") if self.is_gated else ("gate",)
        self.W, self.A, self.B, self.scale = ({c: [] for c in self.cols} for _ in range(4))

    def weight(self, col, q, s):
        """Append the weight s * q to col; q [d_out, d_in] whole numbers, s [d_out, groups of `group` or 32 inputs]."""
        g = self.group or 32
        W = q.double() * s.double().repeat_interleave(g, 1)[:, :self.d_in]
        if not self.group:
            assert torch.equal(W.to(torch.bfloat16).double(), W)
        self.W[col].append((W, q, s))

    def sums(self, col, W=None):
        """The projection's rows in fp64 and which of them there are; W: other weights by slot."""
        W = [w[0] for w in self.W[col]] if W is None else W
        x = self.x.double().repeat_interleave(self.fan, 0)[:self.rows]
        y = x @ W[0].t() if self.adapted else torch.zeros(self.rows, self.d_out, dtype=torch.float64)
        on = torch.full((self.rows,), self.adapted)
        for s in range(self.slots):
            at = torch.from_numpy(np.nonzero(self.ids == s)[0])
            if not self.adapted:
                y[at] = x[at] @ W[s].t()
                on[at] = True
            elif self.rank and len(at):
                y[at] += self.scale[col][s] * (x[at] @ self.A[col][s].double().t() @ self.B[col][s].double().t())
        return y, on


def whole(kind, group, ids, slots, d_in, d_out, rank=0, seed=0, act="silu", fan=1, low=-8, high=7):
    """An exact case.  With adapters: W = D - B A on columns of three very different sizes, so that an output is D x,
    what is left of sums of 2^20 and more: every bit of v counts.  Without: scales of 10 bits."""
    c = Case(kind, group, ids, slots, d_in, d_out, rank, act, fan)
    g = gen(seed + 77)
    G = group or 32
    n = -(-d_in // G)
    ints = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=g)  # noqa: E731
    # one group of large and one of medium columns, one of large gates, whose four inputs are 1; narrow inputs have the last alone
    e = torch.zeros(n, dtype=torch.int64)
    big = {32: 15, 64: 14, 128: 13}[G]
    if rank and n >= 4:
        e[n // 2], e[1] = big, 8
    e[0] = 5 if d_in < 4096 else 6  # (gates of 90 and more: four times 7 of this size above the other columns' spread)
    x_rows = -(-c.rows // fan)
    x = ints(-1, 1, x_rows, d_in) * ints(0, 1, x_rows, d_in)
    x[:, :G] = 0
    x[:, :4] = 1
    c.x = x.to(torch.bfloat16)
    size = torch.ldexp(torch.ones(n), e).repeat_interleave(G)[:d_in].double()
    for col in c.cols:
        A = ints(-3, 3, max(rank, 1), d_in)  # the rank's part of a weight, in its column's size
        A[:, :G] = 0
        of = torch.arange(d_out) % max(rank, 1)
        for s in range(1 if c.adapted else slots):
            D = ints(max(low, -4), min(high, 4), d_out, d_in) if rank else ints(low, high, d_out, d_in)
            D[:, e.repeat_interleave(G)[:d_in] > 0] = 0
            D[:, :4] = 7 if col == "gate" and c.is_gated else 0
            if rank:
                D -= A[of]
            sc = torch.ldexp(torch.ones(d_out, n), e.expand(d_out, n))
            if group and not rank:
                sc = sc * (1 + ints(1, 7, d_out, n) * 2.0 ** -9)
            c.weight(col, D, sc)
        for s in range(slots if rank else 0):
            k = (s % 3) - 1
            c.A[col].append((A.double() * size).to(torch.bfloat16))
            B = torch.zeros(d_out, rank, dtype=torch.float64)
            B[torch.arange(d_out), of] = 2.0 ** -k
            c.B[col].append(B.to(torch.bfloat16))
            c.scale[col].append(2.0 ** k)
        # nothing rounds: what any order of additions can reach, in steps of 2^-10 where scales have 10 bits
        reach = max(float((c.x.double().abs() @ w[0].abs().t()).max()) for w in c.W[col]) * (2 if rank else 1)
        assert reach * (1 if rank or not group else 2 ** 10) < 2 ** 24, reach
    return c


def in_use(kind, group, ids, slots, d_in, d_out, rank=0, seed=0, act="silu", fan=1, low=-8, high=7):
    """A tight case: unit normal x, weights and factors of the sizes that a layer has."""
    c = Case(kind, group, ids, slots, d_in, d_out, rank, act, fan)
    g = gen(seed + 99)
    G = group or 32
    n = -(-d_in // G)
    c.x = torch.randn(-(-c.rows // fan), d_in, generator=g).to(torch.bfloat16)
    for col in c.cols:
        for s in range(1 if c.adapted else slots):
            if group:
                q = torch.randint(low, high + 1, (d_out, d_in), generator=g)
                sc = (torch.rand(d_out, n, generator=g) + 0.5) * d_in ** -0.5 / max(abs(low), abs(high))
                c.weight(col, q, sc)
            else:
                w = (torch.randn(d_out, d_in, generator=g) * d_in ** -0.5).to(torch.bfloat16)
                c.weight(col, w, torch.ones(d_out, n))
        for s in range(slots if rank else 0):
            c.A[col].append((torch.randn(rank, d_in, generator=g) * d_in ** -0.5).to(torch.bfloat16))
            c.B[col].append((torch.randn(d_out, rank, generator=g) * 0.5).to(torch.bfloat16))
            c.scale[col].append(float(np.float32(0.5 + 0.3 * s)))
    return c


def act64(kind, z):
    if kind == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))


def result(c, rounded=lambda col, y: y, W={}):
    """(the call's outputs in fp64, the rows that it writes).  `rounded` and `W` plant mistakes: in a projection's sums, in
    its weights."""
    sums = {}
    for col in c.cols:
        y, on = c.sums(col, W.get(col))
        sums[col] = rounded(col, y)
    if not c.is_gated:
        return sums["gate"], on
    return act64(c.act, sums["gate"]) * sums["up"], on


def once(c):
    """The outputs of an exact case: products of fp32 values rounded to fp32, then to bf16 (fp64 to bf16 in one step
    where nothing is multiplied).  act(g) is g."""
    y, on = c.sums("gate")
    assert torch.equal(y.float().double(), y)
    if c.is_gated:
        assert float(y[on].min()) >= 90
        u, _ = c.sums("up")
        assert torch.equal(u.float().double(), u)
        return (y.float() * u.float()).to(torch.bfloat16), on
    return y.float().to(torch.bfloat16), on


def tight(got, ref):
    """Whether got (bf16 or fp64) is as near to ref (fp64) as a rounding to bf16, by the root of the mean square."""
    rms = lambda t: float(t.double().square().mean().sqrt())  # noqa: E731
    return rms(got.double() - ref) <= 1.01 * rms(ref.to(torch.bfloat16).double() - ref)


def packed(q, s, group, pad=0):
    q = q.to(torch.int32)
    d_out, d_in = q.shape
    Wq = torch.full((d_out, -(-d_in // 32) * 16 + pad), 0xA5, dtype=torch.uint8)
    Wq[:, :d_in // 2] = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8)
    return Wq.cuda(), s.float().contiguous().cuda()


class OnGpu:
    """The library's call of a case; run() builds the segments and makes it."""

    def __init__(self, c, bound=0):
        import adapter_gemv_amd as lg
        self.c, self.keep = c, []
        self.ids = torch.from_numpy(c.ids).cuda()
        x = c.x.cuda()
        self.y = torch.full((max(c.rows, 1), c.d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.seg = lg.Segments(c.rows, max_segments=bound)
        shape = (c.slots, 7)
        ptr = np.zeros((2,) + shape, np.uint64)
        if c.adapted:
            rk, sc = np.zeros(shape, np.int32), np.ones(shape, np.float32)
            for col in c.cols:
                k = MODS.index(col)
                for s in range(c.slots if c.rank else 0):
                    B = torch.zeros(c.d_out, -(-c.rank // 8) * 8, dtype=torch.bfloat16)
                    B[:, :c.rank] = c.B[col][s]
                    for i, t in enumerate((c.A[col][s].cuda(), B.cuda())):
                        ptr[i, s, k] = t.data_ptr()
                        self.keep.append(t)
                    rk[s, k], sc[s, k] = c.rank, c.scale[col][s]
            host = lg.pack_table(ptr[0], ptr[1], rk, sc)
            w = [t for col in c.cols for t in self.weight(col, 0)]
            self.rank = max(c.rank, 1)
            if not c.is_gated:
                self.ios = {"gate": lg.LinearQ4GIO(x, *w, self.y, c.group, d_in=c.d_in)}
                n = lg.linear_q4g_workspace_bytes(c.rows, c.slots, self.rank, c.d_in, 1)
            else:
                self.ios = (lg.GatedQ4GIO(x, *w, self.y, c.group, d_in=c.d_in) if c.group else lg.GatedIO(x, *w, self.y))
                n = lg.gated_workspace_bytes(c.rows, c.slots, self.rank, c.d_in)
        else:
            ld = np.zeros((2,) + shape, np.int64)
            for col in c.cols:
                for s in range(c.slots):
                    w = self.weight(col, s)
                    self.keep.append(w)
                    for i, t in enumerate(w):
                        ptr[i, s, MODS.index(col)], ld[i, s, MODS.index(col)] = t.data_ptr(), t.stride(0)
            host = lg.pack_weights_q4g(ptr[0], ld[0], ptr[1], ld[1]) if c.group else lg.pack_weights(ptr[0], ld[0])
            self.ios = lg.GroupedIO(x, self.y, rows_per_x=c.fan)
            n = lg.workspace_bytes(c.rows, c.slots, 1, 0)
        self.table = torch.from_numpy(host.view(np.uint8).reshape(-1).copy()).cuda()
        self.ws = torch.full((max(n, 16),), 0x7f, dtype=torch.uint8, device="cuda")

    def weight(self, col, s):
        W, q, scales = self.c.W[col][s]
        return packed(q, scales, self.c.group) if self.c.group else (W.to(torch.bfloat16).cuda(),)

    def call(self, rows=None):
        import adapter_gemv_amd as lg
        c, rows = self.c, self.c.rows if rows is None else rows
        at = (rows, self.ids, self.table, c.slots, self.seg, getattr(self, "rank", 0), self.ws)
        if c.kind == "linear":
            lg.linear_layer(self.ios, *at)
        elif c.kind == "gated":
            lg.gated_layer(self.ios, *at, activation=c.act)
        elif c.kind == "grouped":
            lg.grouped_layer_q4g({"gate": self.ios}, rows, self.table, c.slots, self.seg, c.group)
        elif c.group:
            lg.grouped_gated_layer_q4g(self.ios, rows, self.table, c.slots, self.seg, c.group, activation=c.act)
        else:
            lg.grouped_gated_layer(self.ios, rows, self.table, c.slots, self.seg, activation=c.act)

    def run(self):
        import adapter_gemv_amd as lg
        self.y.fill_(float("nan"))
        lg.build_segments(self.ids, self.c.slots, self.seg, self.ws)
        self.call()
        torch.cuda.synchronize()
        return self.y.cpu()
