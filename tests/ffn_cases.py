"""Inputs and 64-bit references of the 4-bit products with stated groups and the
gated half of a feed-forward block (no test functions here).  Everything is
torch on the CPU; the GPU tests move it over.

Tolerances (u = 2^-24, half a step of fp32), beside those of dense_cases:
  * 4-bit sums: a group's is formed as sum (24 + q) x - 24 sum x, every product
    exact in fp32, in 2 G additions of partial sums of at most sum (|q| + 48) |x|,
    each off by 2 u where the matrix cores cut: 2 (2 G + 4) u of that (times the
    scale); the scaled groups are added up in at most n / 32 + 3 steps (n / 32
    where a tile scales every 32 inputs), 2 u each of the sum of magnitudes, and
    the sum's power of two is exact;
  * activation: z sigma(t), t = z (c1 + c3 z^2).  Its derivative is at most 1.13
    in magnitude for both kinds, so an error dz of z is at most 1.13 dz of act.
    t's own roundings are 4 u |t| (three operations and the product with log2 e
    that the exponential makes), of which sigma takes over (1 - sigma) relatively;
    the exponential, the sum and the reciprocal add a unit of the last place each
    (2 u): act_rel = (4 |t| (1 - sigma) + 8) u, doubled for the hardware's
    exponential.  Below t = -87 the exponential passes 2^125 and sigma, at most
    2^-125, may come out as 0;
  * h = act(z) u: 1.13 dz |u| + (|act| + 1.13 dz) du, act_rel |h|, one product.
"""
from __future__ import annotations

import math

import torch

from tests.dense_cases import U

GROUPS = (32, 64, 128)
ACTS = ("silu", "gelu_tanh")


def q4_weight(gen, d_out, d_in, group, pad=0, spad=0):
    """(Wq uint8 [d_out, pitch], Ws fp32 [d_out, groups + spad], W fp64): every value from -8 to 7, junk in what no
    weight lies in."""
    q = torch.randint(-8, 8, (d_out, d_in), generator=gen, dtype=torch.int32)
    pitch = -(-(d_in // 2) // 16) * 16 + pad
    Wq = torch.randint(0, 256, (d_out, pitch), generator=gen, dtype=torch.int32).to(torch.uint8)
    Wq[:, :d_in // 2] = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8)
    n = d_in // group
    Ws = torch.full((d_out, n + spad), float("nan"))
    Ws[:, :n] = (torch.rand(d_out, n, generator=gen) + 0.25) * 0.3 * d_in ** -0.5
    Ws[:, :n][torch.rand(d_out, n, generator=gen) < 0.1] *= -1
    W = q.double() * Ws[:, :n].double().repeat_interleave(group, 1)
    return Wq, Ws, W


def q4_sums(x, W, Ws, group):
    """(y, slack) of the 4-bit product in fp64."""
    x, n = x.double(), W.shape[1]
    mag = x.abs() @ W.abs().t()
    scales = Ws[:, :n // group].double().abs().repeat_interleave(group, 1)
    return x @ W.t(), 2 * (2 * group + 4) * U * (mag + 48 * (x.abs() @ scales.t())) + 2 * (n // 32 + 4) * U * mag


def act64(kind, z):
    """(act, t) in fp64."""
    z = z.double()
    t = z if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(t), t


def gated(kind, z, dz, u, du):
    """(h, slack) from the projections and their slacks."""
    a, t = act64(kind, z)
    h = a * u
    rel = 2 * (4 * t.abs() * torch.sigmoid(-t) + 8) * U
    rel = torch.where(t < -87, torch.zeros_like(rel), rel)
    slack = 1.13 * dz * u.abs() + (a.abs() + 1.13 * dz) * du + (rel + U) * h.abs() + z.abs() * u.abs() * 2.0 ** -125
    return h, slack


# A batch that takes each tile: (kind, the tile's number, its rows and columns of the output, lengths of the segments, or
# rows of a batch over TILE_SLOTS adapters, d_in, d_out).  More than one row tile and column tile, the last of each
# partial, and enough of k that the tile's ring is filled again.
TILE_SLOTS = 5
TILES = [
    ("gated", 0, (16, 32), 21, 1032, 40),
    ("gated", 1, (32, 32), 1030, 1032, 104),
    ("gated", 2, (64, 32), 1030, 1032, 232),
    ("gated", 3, (128, 64), 130, 1032, 5464),
    ("gated", 4, (256, 128), 260, 1032, 11048),
    ("gated_q4g", 0, (4, 16), 5, 1152, 24),
    ("gated_q4g", 1, (4, 16), 6, 8320, 24),
    ("gated_q4g", 2, (4, 32), 130, 1152, 616),
    ("gated_q4g", 3, (16, 16), 700, 2176, 120),
    ("gated_q4g", 4, (16, 32), 1030, 1152, 72),
    ("gated_q4g", 5, (16, 64), 90, 1152, 1176),
    ("gated_q4g", 6, (32, 64), 1030, 1152, 360),
    ("gated_q4g", 7, (64, 128), 100, 1152, 8288),
    ("gated_q4g", 8, (256, 128), 520, 2176, 9496),
    ("grouped_gated", 0, (16, 32), (0, 7, 33), 1032, 40),
    ("grouped_gated", 1, (32, 32), (520, 700, 257), 1032, 72),
    ("grouped_gated", 2, (64, 32), (70, 5, 3), 1032, 2088),
    ("grouped_gated", 3, (128, 64), (200, 15, 5), 1032, 3360),
    ("grouped_gated", 4, (256, 128), (0, 520, 15), 1032, 5040),
    ("grouped_gated_q4g", 0, (4, 16), (3, 7, 5), 1152, 24),
    ("grouped_gated_q4g", 1, (4, 16), (15, 7, 0), 8320, 24),
    ("grouped_gated_q4g", 2, (4, 32), (200, 21, 257), 1152, 168),
    ("grouped_gated_q4g", 3, (16, 16), (300, 21, 70), 2176, 200),
    ("grouped_gated_q4g", 4, (16, 32), (520, 700, 5), 1152, 72),
    ("grouped_gated_q4g", 5, (16, 64), (100, 37, 257), 1152, 280),
    ("grouped_gated_q4g", 6, (32, 64), (3, 37, 15), 1152, 4976),
    ("grouped_gated_q4g", 7, (64, 128), (70, 3, 0), 1152, 8952),
    ("grouped_gated_q4g", 8, (256, 128), (300, 129, 100), 2176, 9032),
    ("grouped_q4g", 0, (4, 32), (5, 3, 7), 1152, 40),
    ("grouped_q4g", 1, (4, 32), (33, 1, 15), 8320, 48),
    ("grouped_q4g", 2, (4, 64), (129, 129, 257), 1152, 296),
    ("grouped_q4g", 3, (16, 32), (700, 520, 127), 2176, 104),
    ("grouped_q4g", 4, (16, 64), (300, 5, 520), 1152, 200),
    ("grouped_q4g", 5, (16, 128), (37, 7, 129), 1152, 2224),
    ("grouped_q4g", 6, (32, 128), (63, 33, 700), 1152, 912),
    ("grouped_q4g", 7, (64, 256), (1, 33, 70), 1152, 13752),
    ("grouped_q4g", 8, (256, 256), (300, 63, 70), 2176, 21648),
    ("linear_q4g", 0, (4, 32), 5, 1152, 40),
    ("linear_q4g", 1, (4, 32), 9, 8320, 40),
    ("linear_q4g", 2, (4, 64), 130, 1152, 1224),
    ("linear_q4g", 3, (16, 32), 1030, 2176, 136),
    ("linear_q4g", 4, (16, 64), 1030, 1152, 136),
    ("linear_q4g", 5, (16, 128), 70, 1152, 5776),
    ("linear_q4g", 6, (32, 128), 1030, 1152, 712),
    ("linear_q4g", 7, (64, 256), 1030, 1152, 1936),
    ("linear_q4g", 8, (256, 256), 520, 2176, 19360),
]
KINDS = ("linear_i8", "grouped", "grouped_i8", "gated", "grouped_gated", "linear_q4g", "grouped_q4g", "gated_q4g",
         "grouped_gated_q4g")


def tile_of(kind, rows, slots, shapes, max_segments=0):
    """(number, rows, columns) of the tile that the library takes for a call of `kind` with these (d_in, d_out)."""
    import ctypes

    import adapter_gemv_amd as lg
    n = len(shapes)
    ints = ctypes.c_int32 * n
    seg = lg._Seg()
    seg.max_segments = max_segments
    f = lg.lib().lora_internal_gemm_tile
    f.restype = ctypes.c_int32
    rt, ct, us = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_double()
    got = f(ctypes.c_int32(KINDS.index(kind)), ctypes.c_int32(rows), ctypes.c_int32(slots), seg,
            ints(*[s[0] for s in shapes]), ints(*[s[1] for s in shapes]), ctypes.c_int32(n), ctypes.byref(rt),
            ctypes.byref(ct), ctypes.byref(us))
    assert got >= 0
    return got, rt.value, ct.value
