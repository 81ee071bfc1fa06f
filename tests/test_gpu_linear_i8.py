"""GPU tests of the int8 base projection with the adapter delta
(lora_linear_layer_i8) against the 64-bit definition."""
import numpy as np
import pytest

from tests.dense_cases import (LINEAR_SLOTS, LINEAR_TILES, MODS, U, base_i8, bf16, close, close_range, delta, extreme_rows,
                               extreme_scales, gen, ids_of, int8_weight, quantise_rows, tile_of)
from tests.parity import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import adapter_gemv_amd as lg  # noqa: E402


@pytest.fixture(autouse=True)
def _name_case(request):
    note(request.node.nodeid)


class Run:
    """A batch with adapters and int8 base weights, on the CPU and on the GPU."""

    def __init__(self, rows, slots, shapes, ranks, kind="mixed", seed=0, fmt="bf16", strided=False, x_std=1.0,
                 bound=False):
        g = gen(seed + 1)
        self.rows, self.slots, self.shapes = rows, slots, shapes
        self.ids = ids_of(kind, rows, slots, seed)
        ranks = [ranks] * slots if isinstance(ranks, int) else [ranks[s % len(ranks)] for s in range(slots)]
        self.max_rank = max(max(ranks), 1)
        pad = 16 if strided else 0
        self.cpu, self.dev, self.keep = {}, {}, []
        A_p = np.zeros((slots, 7), np.uint64)
        B_p, rk = A_p.copy(), np.zeros((slots, 7), np.int32)
        sc, fm = np.ones((slots, 7), np.float32), np.zeros((slots, 7), np.int32)
        xs = {}
        for m, (di, do, share) in shapes.items():
            if share not in xs:
                full = bf16(g, rows, di + pad, std=x_std)
                xs[share] = (full, full.cuda())
            Wq, Ws = int8_weight(g, do, di)
            c = {"x": xs[share][0][:, :di], "Wq": Wq, "Ws": Ws, "A": [], "B": [], "scale": []}
            y = torch.full((rows, do + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
            self.dev[m] = lg.LinearI8IO(xs[share][1], Wq.cuda(), Ws.cuda(), y, d_in=di, d_out=do)
            col = MODS.index(m)
            for s in range(slots):
                r = ranks[s]
                A, B = bf16(g, r, di, std=0.1), bf16(g, do, r, std=0.1)
                scale = float(np.float32(0.25 + 0.5 * ((s * 7 + col) % 5)))
                if r and (fmt == "int8" or (fmt == "both" and s % 2)):
                    A, B, pa, pb = self.int8_factors(A, B)
                    fm[s, col] = lg.FORMAT_INT8_ROWS
                else:
                    ldb = -(-max(r, 1) // 8) * 8
                    Bp = torch.zeros(do, ldb, dtype=torch.bfloat16)
                    Bp[:, :r] = B
                    pa, pb = A.cuda(), Bp.cuda()
                self.keep += [pa, pb]
                A_p[s, col], B_p[s, col] = (pa.data_ptr(), pb.data_ptr()) if r else (0, 0)
                rk[s, col], sc[s, col] = r, scale
                c["A"].append(A)
                c["B"].append(B)
                c["scale"].append(scale)
            self.cpu[m] = c
        self.table_host = lg.pack_table(A_p, B_p, rk, sc, fm)
        self.seg = lg.Segments(rows, max_segments=lg.segment_bound(self.ids, slots) if bound else 0)
        n = lg.linear_i8_workspace_bytes(rows, slots, self.max_rank, sum(s[0] for s in shapes.values()), len(shapes))
        self.ws = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
        self.dids = torch.from_numpy(self.ids).cuda()
        self.upload()

    def upload(self):
        self.table = torch.from_numpy(self.table_host.view(np.uint8).reshape(-1).copy()).cuda()

    def int8_factors(self, A, B):
        def q(t):
            t = t.float()
            s = t.abs().amax(1) / 127 + 1e-6
            return torch.round(t / s[:, None]).clamp(-127, 127).to(torch.int8), s

        def block(qv, s, ld):
            n4 = -(-s.numel() // 4) * 4
            sc = torch.zeros(n4)
            sc[:s.numel()] = s
            v = torch.zeros(qv.shape[0], ld, dtype=torch.int8)
            v[:, :qv.shape[1]] = qv
            return torch.cat([sc.view(torch.uint8), v.view(torch.uint8).reshape(-1)]).cuda()

        qa, sa = q(A)
        qb, sb = q(B)
        return (qa.double() * sa.double()[:, None], qb.double() * sb.double()[:, None],
                block(qa, sa, -(-A.shape[1] // 16) * 16), block(qb, sb, -(-max(B.shape[1], 1) // 16) * 16))

    def args(self):
        return (self.dev, self.rows, self.dids, self.table, self.slots, self.seg, self.max_rank, self.ws)

    def launch(self, phases=False):
        lg.build_segments(self.dids, self.slots, self.seg, self.ws)
        if phases:
            lg.linear_layer(*self.args(), _fn="lora_linear_shrink")
            lg.linear_layer(*self.args(), _fn="lora_linear_expand")
        else:
            lg.linear_layer(*self.args())

    def out(self):
        return {m: io.y[:, :io.d_out].clone() for m, io in self.dev.items()}

    def run(self, phases=False):
        for io in self.dev.values():
            io.y.fill_(float("nan"))
        self.launch(phases)
        torch.cuda.synchronize()
        return self.out()

    def reference(self, m, skip=()):
        c = self.cpu[m]
        di = self.shapes[m][0]
        y, slack = base_i8(c["x"], c["Wq"][:, :di], c["Ws"])
        for s in range(self.slots):
            at = np.nonzero(self.ids == s)[0]
            if len(at) == 0 or s in skip or c["A"][s].shape[0] == 0:
                continue
            d, sl = delta(c["x"][at], c["A"][s], c["B"][s], c["scale"][s])
            y[at] += d
            slack[at] += sl
        return y, slack

    def check(self, got=None, skip=()):
        got = self.run() if got is None else got
        for m in self.shapes:
            ref, slack = self.reference(m, skip)
            close(got[m], ref, slack, m)


def qkv(d, kv):
    return {"q": (d, d, "a"), "k": (d, kv, "a"), "v": (d, kv, "a")}


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 129, 300])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_rows(rows, kind):
    Run(rows, 5, qkv(264, 72), (16, 0, 64, 5, 33), kind, seed=rows).check()


@pytest.mark.parametrize("d_in,d_out", [(8, 8), (16, 24), (40, 8), (120, 136), (128, 128), (136, 264), (512, 32), (520, 40),
                                        (1032, 72), (2056, 520), (4104, 16)])
@pytest.mark.parametrize("rows", [1, 20, 40, 100, 200])
def test_widths(d_in, d_out, rows):
    Run(rows, 3, {"o": (d_in, d_out, "o")}, (8, 24), "mixed", seed=d_in + d_out).check()


@pytest.mark.parametrize("rank", [1, 7, 8, 16, 31, 32, 40, 64])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "both"])
@pytest.mark.parametrize("rows", [3, 50, 140])
def test_ranks_and_formats(rank, fmt, rows):
    Run(rows, 4, {"gate": (136, 200, "m"), "down": (200, 136, "d")}, rank, "mixed", seed=rank, fmt=fmt).check()


@pytest.mark.parametrize("rows", [24, 150, 2600])
def test_distinct_adapter_per_row(rows):
    slots = min(rows, 150)
    Run(rows, slots, {"k": (264, 136, "a"), "up": (264, 264, "m")}, (64, 16, 8), "distinct", seed=3).check()


@pytest.mark.parametrize("kind,fmt", [("runs", "bf16"), ("mixed", "both"), ("none", "bf16"), ("one", "int8")])
def test_largest_tile(kind, fmt):
    # 4101 rows x 4104 outputs: enough 256 x 256 tiles for every compute unit, the last ones partial
    Run(4101, 9, {"q": (136, 4104, "a")}, (16, 64, 0, 33), kind, seed=11, fmt=fmt).check()


def test_whole_layer():
    shapes = {"q": (520, 520, "a"), "k": (520, 72, "a"), "v": (520, 72, "a"), "o": (520, 520, "o"),
              "gate": (520, 1032, "m"), "up": (520, 1032, "m"), "down": (1032, 520, "d")}
    Run(37, 19, shapes, (5, 16, 64), "mixed", seed=2).check()


def test_strided():
    Run(45, 4, {"q": (264, 136, "a"), "o": (136, 264, "o")}, (16, 8), "mixed", seed=4, strided=True).check()


def test_base_only_and_no_targeted_projection():
    Run(30, 4, {"q": (264, 136, "a")}, 8, "none", seed=5).check()
    Run(30, 4, {"q": (264, 136, "a")}, 0, "mixed", seed=5).check()


@pytest.mark.parametrize("rows", [1, 30, 70, 130, 260])
def test_base_is_exact(rows):
    # no adapters: y = bf16((acc * s) * Ws), every step of which the definition fixes to the bit
    r = Run(rows, 2, {"q": (1032, 264, "a")}, 8, "none", seed=rows)
    got = r.run()["q"]
    c = r.cpu["q"]
    q, _ = quantise_rows(c["x"])
    acc = (q.double() @ c["Wq"][:, :1032].double().t()).float()
    s = c["x"].float().abs().amax(1) / 127.0
    want = ((acc * s[:, None]) * c["Ws"][None]).to(torch.bfloat16)
    assert torch.equal(got.cpu(), want)


def test_ties_and_extremes_of_the_quantiser():
    # amax 1 and 127 put many values on ties of 127 x / amax; amax at the ends of the type; a zero row
    d = 264
    r = Run(9, 1, {"q": (d, 64, "a")}, 8, "none", seed=1)
    x = torch.zeros(9, d)
    x[0] = (torch.arange(d) % 255 - 127).float() / 254
    x[0, 5] = 1.0
    x[1] = (torch.arange(d) % 255 - 127).float() / 2
    x[1, 7] = -127.0
    x[2] = torch.linspace(-3e38, 3e38, d)
    x[3] = torch.linspace(-1e-38, 1e-38, d)
    x[4] = 0.0
    x[5] = -1.0
    x[6, 3] = 2.0 ** -126
    x[7] = torch.linspace(-1, 1, d) * 2.0 ** -20
    x[8] = torch.randn(d, generator=gen(3)) * 50
    x = x.to(torch.bfloat16)
    r.cpu["q"]["x"] = x
    r.dev["q"].x = x.cuda()
    r.check()


@pytest.mark.parametrize("copies", [1, 5])
def test_quantiser_over_every_pair_of_significands(copies):
    # row a: amax with significand 128 + a, every significand at 8 magnitudes below it; W is the identity, so the
    # outputs are the quantised values times the scale (5 copies: rows past the quantiser's registers)
    sig = torch.arange(128, 256).double()
    cols = torch.cat([sig * 2.0 ** -k for k in range(1, 9)])                    # all below 128
    x = torch.stack([torch.cat([cols * (1 if a % 2 else -1), torch.tensor([float(a)]).double()]) for a in range(128, 256)])
    x = torch.nn.functional.pad(x, (0, 7))                                      # 1032 inputs
    d = x.shape[1]
    r = Run(128, 1, {"q": (d * copies, d, "a")}, 8, "none", seed=7)
    xb = x.repeat(1, copies).to(torch.bfloat16)
    assert torch.equal(xb[:, :d].double(), x)                                    # every value is a bf16
    r.cpu["q"]["x"] = xb
    r.dev["q"].x = xb.cuda()
    W = torch.zeros(d, -(-d * copies // 16) * 16, dtype=torch.int8)
    W[torch.arange(d), torch.arange(d) + d * (copies - 1)] = 1                  # the last copy
    r.dev["q"].Wq.copy_(W)
    r.dev["q"].Ws.fill_(1.0)
    got = r.run()["q"].cpu()
    amax = x.abs().amax(1, keepdim=True)
    want = (torch.round(127.0 * x / amax).float() * (amax.float() / 127.0)).to(torch.bfloat16)
    assert torch.equal(got, want)


def test_non_finite_rows_stay_alone():
    r = Run(40, 3, {"q": (264, 136, "a")}, 0, "none", seed=8)
    x = r.cpu["q"]["x"].clone()
    x[3, 17] = float("inf")
    x[9, 0] = float("nan")
    x[20, 263] = float("-inf")
    r.cpu["q"]["x"] = x
    r.dev["q"].x = x.cuda()
    got = r.run()
    r.check(got)
    assert set(torch.nonzero(torch.isnan(got["q"]).any(1))[:, 0].tolist()) == {3, 9, 20}


@pytest.mark.parametrize("rows", [16, 60, 200])
def test_a_broken_adapter_reaches_its_own_rows_only(rows):
    r = Run(rows, 6, {"q": (136, 72, "a")}, 16, "mixed", seed=21)
    for s, v in ((1, float("nan")), (4, float("inf"))):  # the B of two adapters
        t = r.keep[2 * s + 1]
        t[5, 3] = v
    got = r.run()["q"].cpu()
    sick = np.isin(r.ids, (1, 4))
    assert not torch.isfinite(got[sick][:, 5]).any()
    ref, slack = r.reference("q")
    close(got[~sick], ref[~sick], slack[~sick], "healthy rows")
    other = np.arange(72) != 5
    close(got[sick][:, other], ref[sick][:, other], slack[sick][:, other], "other outputs")


def test_bad_entries_count_and_leave_the_base():
    r = Run(50, 6, {"q": (136, 72, "a"), "o": (136, 72, "o")}, 16, "mixed", seed=23)
    t = r.table_host
    t["rank"][1, 0] = 17          # above max_rank
    t["A"][2, 0] = 0
    t["B"][3, 0] += 8             # misaligned
    t["format"][4, 3] = 9
    r.upload()
    got = r.run()
    present = set(r.ids.tolist())
    bad_rows = int(((r.ids >= r.slots)).sum())
    want = bad_rows + sum(s in present for s in (1, 2, 3, 4))
    assert int(r.seg.status.item()) == want
    ref, slack = r.reference("q", skip=(1, 2, 3))
    close(got["q"], ref, slack, "q")
    ref, slack = r.reference("o", skip=(4,))
    close(got["o"], ref, slack, "o")


def test_segment_bound():
    r = Run(64, 40, {"q": (136, 72, "a")}, 16, "mixed", seed=25, bound=True)
    r.check()
    r.seg.max_segments = 7  # keeps the lowest 7 slots; the others' rows get the base alone
    dropped = sorted(set(i for i in r.ids.tolist() if 0 <= i < r.slots))[7:]
    r.check(skip=dropped)


def test_parts_equal_the_whole_and_bits_repeat():
    r = Run(70, 9, qkv(264, 136), (16, 64), "mixed", seed=31)
    a, b, c = r.run(), r.run(phases=True), r.run()
    for m in a:
        assert torch.equal(a[m], b[m]) and torch.equal(a[m], c[m])


def test_rows_past_the_batch_and_columns_past_d_out_stay():
    r = Run(21, 3, {"q": (136, 72, "a")}, 8, "mixed", seed=33)
    y = torch.full((32, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    r.dev["q"].y = y
    r.launch()
    torch.cuda.synchronize()
    assert bool((y[21:] == 7).all()) and bool((y[:, 72:] == 7).all())
    ref, slack = r.reference("q")
    close(y[:21, :72], ref, slack, "q")


def test_segments_of_a_longer_batch_stay_inside_this_one():
    # a breach of the precondition (segments and rows belong together): what is written stays inside the batch
    r = Run(100, 5, {"q": (136, 72, "a")}, 8, "mixed", seed=35)
    lg.build_segments(r.dids, r.slots, r.seg, r.ws)
    y = torch.full((100, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    r.dev["q"].y = y
    r.rows = 70
    lg.linear_layer(*r.args())
    torch.cuda.synchronize()
    assert bool((y[70:] == 7).all()) and bool(torch.isfinite(y).all())


def test_zero_rows():
    r = Run(4, 2, {"q": (136, 72, "a")}, 8, "mixed", seed=34)
    r.rows = 0
    got = r.run()["q"]
    assert bool(torch.isnan(got).all())


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_graph_replays(rows):
    r = Run(rows, 6, qkv(264, 136), (16, 8), "mixed", seed=41)
    want = r.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.launch()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.launch()
    for k in range(4):
        for io in r.dev.values():
            io.y.fill_(float("nan"))
        r.ws.fill_(0x7f)
        graph.replay()
        torch.cuda.synchronize()
        got = r.out()
        for m in got:
            assert torch.equal(got[m], want[m]), (k, m)
        eager = r.run()
        for m in got:
            assert torch.equal(eager[m], want[m]), (k, m)
    # new contents in the same buffers: the graph follows them
    x = bf16(gen(99), *r.cpu["q"]["x"].shape)
    for m in r.dev:
        r.cpu[m]["x"] = x
    r.dev["q"].x.copy_(x)
    ids = ids_of("mixed", rows, 6, 77)
    r.ids = ids
    r.dids.copy_(torch.from_numpy(ids))
    graph.replay()
    torch.cuda.synchronize()
    r.check(r.out())


def test_two_streams_with_their_own_workspaces():
    a = Run(33, 4, qkv(520, 136), (16, 8), "mixed", seed=51)
    b = Run(150, 4, qkv(520, 136), (64, 8), "mixed", seed=52)
    wa, wb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.launch()
        with torch.cuda.stream(s2):
            b.launch()
    torch.cuda.synchronize()
    for r, want in ((a, wa), (b, wb)):
        got = r.out()
        for m in got:
            assert torch.equal(got[m], want[m])


@pytest.mark.parametrize("d_in", [8200, 28672])
def test_long_rows(d_in):
    # past the quantiser's registers; the strong channel fixes the scale
    r = Run(5, 2, {"down": (d_in, 40, "d")}, 16, "mixed", seed=61)
    x = r.cpu["down"]["x"].clone()
    x[:, d_in - 1] = 37.0
    r.cpu["down"]["x"] = x
    r.dev["down"].x = x.cuda()
    r.check()


def test_most_inputs_and_largest_sums():
    # 131072 inputs, all products 127 * -128: the sum, -2^31 + 2^24, fits int32
    d_in = lg.I8_MAX_IN
    r = Run(2, 1, {"down": (d_in, 16, "d")}, 8, "none", seed=62)
    x = torch.ones(2, d_in, dtype=torch.bfloat16)
    r.cpu["down"]["x"] = x
    r.dev["down"].x = x.cuda()
    r.cpu["down"]["Wq"][:] = -128
    r.dev["down"].Wq.fill_(-128)
    r.check()


@pytest.mark.parametrize("rows", [1, 37, 300])
def test_workspace_is_not_overrun(rows):
    shapes = {"q": (1032, 72, "a"), "k": (1032, 40, "a"), "o": (8, 264, "o"), "down": (4104, 16, "d")}
    r = Run(rows, 5, shapes, (5, 64), "mixed", seed=63)
    n = r.ws.numel()
    big = torch.full((n + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    r.ws = big[:n]
    r.check()
    assert bool((big[n:] == 0x5a).all())


@pytest.mark.parametrize("rows,upto", [(100, 70), (40, 30), (300, 200), (700, 400)])
@pytest.mark.parametrize("bound", [False, True])
def test_rows_past_the_batch_in_segments_that_fit_touch_nothing(rows, upto, bound):
    stray_rows(rows, upto, bound, {"q": (136, 200, "a"), "o": (72, 40, "o")})


@pytest.mark.parametrize("tile,rows,upto,d_out", [((128, 128), 300, 200, 8200), ((256, 256), 1300, 900, 12296)])
def test_rows_past_the_batch_touch_nothing_on_tiles_that_store_whole_lines(tile, rows, upto, d_out):
    assert tile_of("linear_i8", upto, 5, [(136, d_out)]) == tile
    stray_rows(rows, upto, False, {"q": (136, d_out, "a")})


def stray_rows(rows, upto, bound, shapes):
    # segments of a longer batch: every row of this one gets its own result or none, the delta only from a segment that
    # ends inside the batch, and rows past it are left alone
    r = Run(rows, 5, shapes, 8, "mixed", seed=36, bound=bound)
    lg.build_segments(r.dids, r.slots, r.seg, r.ws)
    _, offs, slots, _ = r.seg.host()
    fit = [int(s) for s, end in zip(slots, offs[1:]) if end <= upto]
    assert any((r.ids[upto:] == s).any() for s in fit)  # stray rows are there
    for io in r.dev.values():
        io.y.fill_(7.0)
    r.rows = upto
    lg.linear_layer(*r.args())
    torch.cuda.synchronize()
    for m, y in r.out().items():
        assert bool((y[upto:] == 7).all()), m
        written = torch.nonzero(~(y[:upto] == 7).all(1))[:, 0].cpu()
        assert len(written) >= upto // 2
        ref, slack = r.reference(m, skip=[s for s in range(r.slots) if s not in fit])
        close(y[written], ref[written], slack[written], m)


def test_rows_and_scales_at_the_ends_of_the_type():
    # sums of 2^23 under row scales from 2^-140 to 2^121 and output scales from 2^-121 to 2^98: finite wherever the
    # definition is (the smallest scales lie below the documented range, where sums as large as these are still safe).
    # The base rounds four times: 4 u (extreme_rows and _scales hold no value that is not exact)
    d = 264
    r = Run(12, 1, {"q": (d, 64, "a")}, 8, "none", seed=1)
    c = r.cpu["q"]
    c["x"], c["Ws"] = extreme_rows(d), extreme_scales(c["Ws"])
    r.dev["q"].x, r.dev["q"].Ws = c["x"].cuda(), c["Ws"].cuda()
    ref, _ = r.reference("q")
    assert int((ref.abs() < 2.0 ** 127).sum()) > ref.numel() // 2 and int((ref.abs() > 2.0 ** 100).sum()) > 100
    close_range(r.run()["q"], ref, 4 * U, "q")


@pytest.mark.parametrize("rows", [40, 200])
def test_non_finite_rows_among_rows_with_adapters(rows):
    r = Run(rows, 3, {"q": (264, 136, "a")}, (16, 64, 5), "mixed", seed=9)
    x = r.cpu["q"]["x"].clone()
    sick = [3, 9, 20, rows - 1]
    for b, v in zip(sick, ("inf", "nan", "-inf", "nan")):
        x[b, 17 + b] = float(v)
    assert sum(r.ids[b] in (0, 1, 2) for b in sick) >= 2
    r.cpu["q"]["x"] = x
    r.dev["q"].x = x.cuda()
    got = r.run()
    r.check(got)
    assert set(torch.nonzero(torch.isnan(got["q"]).any(1))[:, 0].tolist()) == set(sick)


@pytest.mark.parametrize("copies", [8, 24, 64])
def test_quantiser_over_the_significands_of_amaxs_own_power_of_two(copies):
    # row a: amax with significand 128 + a and every significand up to it at its own power of two (q from 64 to 127, where
    # a quotient comes nearest to a tie: 254 beside 255); W is the identity.  8 copies: a wave a row; 24: past its
    # registers; 64: a block a row and past its registers
    sig = torch.arange(128, 256).double()
    x = torch.stack([torch.where(sig <= a, sig, torch.zeros(128).double()) * (1 if a % 2 else -1) for a in range(128, 256)])
    x = torch.cat([x, sig[:, None], torch.zeros(128, 7).double()], 1)            # 136 inputs, the largest is a
    d = x.shape[1]
    r = Run(128, 1, {"q": (d * copies, d, "a")}, 8, "none", seed=7)
    xb = x.repeat(1, copies).to(torch.bfloat16)
    assert torch.equal(xb[:, :d].double(), x)                                    # every value is a bf16
    r.cpu["q"]["x"] = xb
    r.dev["q"].x = xb.cuda()
    W = torch.zeros(d, -(-d * copies // 16) * 16, dtype=torch.int8)
    W[torch.arange(d), torch.arange(d) + d * (copies - 1)] = 1                   # the last copy
    r.dev["q"].Wq.copy_(W)
    r.dev["q"].Ws.fill_(1.0)
    got = r.run()["q"].cpu()
    amax = x.abs().amax(1, keepdim=True)
    want = (torch.round(127.0 * x / amax).float() * (amax.float() / 127.0)).to(torch.bfloat16)
    assert torch.equal(got, want)


@pytest.mark.parametrize("tile,rows,d_in,d_out", LINEAR_TILES)
@pytest.mark.parametrize("ranks,kind,fmt", [((16, 0, 8, 5, 32), "mixed", "bf16"), ((64, 0, 33, 40, 5), "runs", "both"),
                                            ((64, 40, 17, 64, 33), "mixed", "bf16"), ((32, 8, 24, 1, 16), "runs", "int8")])
def test_each_tile(tile, rows, d_in, d_out, ranks, kind, fmt):
    # every kernel of the int8 base, its ring filled again and its edges partial; ranks up to 32 and above are two of them
    assert tile_of("linear_i8", rows, LINEAR_SLOTS, [(d_in, d_out)]) == tile
    Run(rows, LINEAR_SLOTS, {"q": (d_in, d_out, "a")}, ranks, kind, seed=rows + d_in, fmt=fmt).check()


def test_whole_layer_of_decode_rows():
    # every projection on the 128-row tile, as a whole layer's decode batch takes it
    shapes = {"q": (1032, 1032, "a"), "k": (1032, 128, "a"), "v": (1032, 128, "a"), "o": (1032, 1032, "o"),
              "gate": (1032, 4128, "m"), "up": (1032, 4128, "m"), "down": (4128, 1032, "d")}
    assert tile_of("linear_i8", 130, 150, [s[:2] for s in shapes.values()]) == (128, 128)
    Run(130, 150, shapes, (64, 8, 16, 8), "distinct", seed=3).check()
