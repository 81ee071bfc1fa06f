"""Inputs and 64-bit references of the int8 base projection and the grouped
products (no test functions here).  Everything is torch on the CPU; the GPU
tests move it over.

Tolerances (u = 2^-24, half a step of fp32):
  * the output's rounding: half a bf16 step, 2^-8 of |y|;
  * int8 base: the int32 sum is exact; its conversion, the row scale (one
    division) and the two products round four times: 4 u |base|;
  * bf16 products: n terms added in fp32 in some order err by at most n u times
    the sum of their magnitudes (2 n u: an adder of the matrix cores may cut
    instead of rounding);
  * delta: the same for A x (n = d_in) and B v (n = rank), and v enters the
    second product as two bf16 pieces, 2^-16 of its magnitude at most.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
BF = 2.0 ** -8
MODS = ("q", "k", "v", "o", "gate", "up", "down")


def quantise_rows(x):
    """(q int64, s fp64) of bf16 rows, exact quotients rounded half to even."""
    x = x.double()
    amax = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64)
    bad = ~torch.isfinite(x).all(1)
    safe = torch.where((amax > 0) & ~bad, amax, torch.ones_like(amax))
    q = torch.round(127.0 * torch.where(bad[:, None], torch.zeros_like(x), x) / safe[:, None])
    s = amax / 127.0
    s[bad] = float("nan")
    return q.long(), s


def close(got, ref, slack, what):
    """got (bf16 values), ref and slack fp64 [rows, n]: |got - ref| <= 2^-8 |ref| + slack, NaN where ref is."""
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    err = (got - ref).abs()[~nan]
    tol = (BF * ref.abs() + slack)[~nan] + 1e-30
    bad = int((err > tol).sum())
    if bad:
        i = int((err - tol).argmax())
        raise AssertionError(f"{what}: {bad} of {err.numel()} out of tolerance; worst {float(err[i])} > {float(tol[i])}")


def base_i8(x, Wq, Ws):
    """(y, slack) of the int8 product in fp64 (integer sums exact below 2^53)."""
    q, s = quantise_rows(x)
    acc = torch.matmul(q.double(), Wq.double().t())
    y = acc * s[:, None] * Ws.double()[None]
    y[torch.isnan(s)] = float("nan")
    return y, 4 * U * y.abs().nan_to_num()


def delta(x, A, B, scale):
    """(delta, slack) of one adapter on rows x; A [r, d_in], B [d_out, r] fp64 values."""
    x, A, B = x.double(), A.double(), B.double()
    v = x @ A.t()
    va = x.abs() @ A.abs().t()
    r, d_in = A.shape
    d = scale * (v @ B.t())
    mag = abs(scale) * (va @ B.abs().t())
    return d, (2 * (d_in + r + 2) * U + 2.0 ** -16) * mag


def grouped_bf16(x, W):
    x, W = x.double(), W.double()
    return x @ W.t(), 2 * (W.shape[1] + 2) * U * (x.abs() @ W.abs().t())


def int8_weight(gen, d_out, d_in, pitch=None):
    """(Wq padded to a multiple of 16 with junk in the padding, Ws)."""
    pitch = -(-d_in // 16) * 16 if pitch is None else pitch
    Wq = torch.randint(-127, 128, (d_out, pitch), generator=gen, dtype=torch.int32).to(torch.int8)
    Wq[:, :2] = -128  # the type's lowest value too
    Ws = (torch.rand(d_out, generator=gen) + 0.5) / 127 * d_in ** -0.5
    return Wq, Ws


def bf16(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def ids_of(kind, n, slots, seed):
    r = np.random.RandomState(seed)
    if kind == "distinct":
        ids = r.permutation(max(n, slots))[:n] % slots
    elif kind == "runs":
        cuts = np.sort(r.randint(0, n + 1, max(slots - 1, 0)))
        ids = np.searchsorted(cuts, np.arange(n), side="right")
        ids = r.permutation(slots)[np.minimum(ids, slots - 1)]
    elif kind == "one":
        ids = np.full(n, slots - 1)
    elif kind == "none":
        ids = np.full(n, -1)
    else:  # mixed: uniform, some base only, some out of range
        ids = r.randint(0, slots, n)
        ids[r.rand(n) < 0.15] = -1
        ids[r.rand(n) < 0.05] = slots + 3
    return ids.astype(np.int32)


def close_range(got, ref, rel, what):
    """got (bf16 values) against ref (fp64) over the whole range of the type: |got - ref| <= (2^-8 + rel) |ref| plus half
    a step of the smallest values (2^-134, and 2^-150 where fp32 rounds one to its own); infinite where ref rounds past
    the largest value, NaN where ref is."""
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    got, ref = got[~nan], ref[~nan]
    edge = 2.0 ** 128 - 2.0 ** 119  # half a step above the largest value
    over = ref.abs() > edge * (1 + rel)
    assert torch.equal(got[over], ref[over].sign() * float("inf")), f"{what}: not infinite past the type"
    sure = ref.abs() < edge * (1 - rel)
    err, tol = (got - ref)[sure].abs(), (BF + rel) * ref[sure].abs() + 2.0 ** -134 + 2.0 ** -150
    bad = int((~(err <= tol)).sum())
    assert bad == 0, f"{what}: {bad} of {err.numel()} out of tolerance; largest error {float(err.max())}"


def extreme_rows(d):
    """[12, d] bf16 rows at both ends of the type, every value finite."""
    ramp = torch.linspace(-1, 1, d).double()
    top, low = 3e38, 2.0 ** -133  # near the largest value; the smallest of all
    one = torch.zeros(d).double()
    one[d // 3] = 1.0
    rows = [ramp * top, ramp * 1e36, ramp * 1e30, one * top, ramp, torch.zeros(d).double(), ramp * 1e-30, ramp * 1e-38,
            ramp * 2.0 ** -126, ramp * 2.0 ** -129, one * low, -one * low * 3]
    x = torch.stack(rows).to(torch.bfloat16)
    assert bool(torch.isfinite(x).all()) and float(x[0].abs().max()) > 2.9e38 and float(x[10].abs().max()) == low
    return x


def extreme_scales(Ws):
    """The scales of the outputs by powers of two, exactly, so that products of either end meet scales of the other:
    a quarter of the outputs each at 1, 2^60, 2^-60 and (half of them) 2^110 or 2^-110."""
    n = Ws.numel()
    e = torch.tensor([0, 60, -60, 110, 0, 60, -60, -110])[torch.arange(n) % 8]
    out = torch.ldexp(Ws, e)
    assert bool(torch.isfinite(out).all()) and bool((out.abs() > 2.0 ** -126).all())
    return out


# The tile (rows, columns) of a product and a batch that takes it: more than one row tile and column tile, the last of
# each partial, and enough of k that every place of the tile's ring is filled again.
LINEAR_TILES = [((16, 64), 37, 2056, 264), ((32, 64), 260, 1032, 1032), ((64, 64), 100, 1032, 4104),
                ((128, 96), 520, 1032, 4104), ((128, 128), 260, 1032, 8200), ((256, 256), 520, 1032, 16392),
                ((256, 256), 1030, 2056, 8200)]
GROUPED_TILES = [((16, 64), (21, 1, 15), 2056, 264), ((32, 64), (100, 31, 129), 1032, 1032),
                 ((64, 64), (100, 31, 129), 1032, 2056), ((128, 96), (127, 4, 129), 1032, 6152),
                 ((128, 128), (127, 4, 129), 1032, 8200), ((256, 256), (300, 1, 219), 1032, 12296),
                 ((256, 256), (0, 1030, 600), 2056, 8200)]
LINEAR_SLOTS = 5


def tile_of(kind, rows, slots, shapes, max_segments=0):
    """(rows, columns) of the tile that the library takes for a call of `kind` ("linear_i8", "grouped" or "grouped_i8") with
    these (d_in, d_out)."""
    import ctypes

    import adapter_gemv_amd as lg
    n = len(shapes)
    ints = ctypes.c_int32 * n
    seg = lg._Seg()
    seg.max_segments = max_segments
    f = lg.lib().lora_internal_gemm_tile
    f.restype = ctypes.c_int32
    rt, ct, us = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_double()
    got = f(ctypes.c_int32(["linear_i8", "grouped", "grouped_i8"].index(kind)), ctypes.c_int32(rows), ctypes.c_int32(slots),
            seg, ints(*[s[0] for s in shapes]), ints(*[s[1] for s in shapes]), ctypes.c_int32(n), ctypes.byref(rt),
            ctypes.byref(ct), ctypes.byref(us))
    assert got >= 0
    return rt.value, ct.value
