"""GPU tests of the dense products grouped by slot (lora_grouped_layer,
lora_grouped_layer_i8) against the 64-bit definition."""
import numpy as np
import pytest

from tests.dense_cases import (GROUPED_TILES, MODS, U, base_i8, bf16, close, close_range, extreme_rows, extreme_scales, gen,
                               grouped_bf16, ids_of, int8_weight, tile_of)
from tests.parity import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import adapter_gemv_amd as lg  # noqa: E402

FORMS = [False, True]


@pytest.fixture(autouse=True)
def _name_case(request):
    note(request.node.nodeid)


class Run:
    def __init__(self, int8, ids, slots, shapes, fan=1, seed=0, pad=0, bound=0, none=()):
        g = gen(seed + 1)
        self.int8, self.ids, self.slots, self.shapes, self.fan = int8, np.asarray(ids, np.int32), slots, shapes, fan
        self.rows = rows = len(ids)
        self.none = set(none)
        self.cpu, self.dev, self.keep = {}, {}, {}
        t = np.zeros((slots, 7), lg.WEIGHT_ENTRY_DTYPE)
        xs = {}
        for m, (di, do, share) in shapes.items():
            if share not in xs:
                full = bf16(g, max(-(-rows // fan), 1), di + pad)
                xs[share] = (full, full.cuda())
            c = {"x": xs[share][0][:, :di], "W": [], "Ws": []}
            y = torch.full((max(rows, 1), do + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            self.dev[m] = lg.GroupedIO(xs[share][1], y, d_in=di, d_out=do, rows_per_x=fan)
            for s in range(slots):
                if int8:
                    W, Ws = int8_weight(g, do, di, -(-di // 16) * 16 + pad)
                    dws = Ws.cuda()
                else:
                    W, Ws, dws = bf16(g, do, di + pad, std=di ** -0.5), None, None
                dw = W.cuda()
                self.keep[m, s] = (dw, dws)
                c["W"].append(W[:, :di])
                c["Ws"].append(Ws)
                if s not in self.none:
                    col = MODS.index(m)
                    t["W"][s, col], t["ldw"][s, col] = dw.data_ptr(), dw.stride(0)
                    t["Ws"][s, col] = dws.data_ptr() if int8 else 0
            self.cpu[m] = c
        self.host = t
        self.seg = lg.Segments(rows, max_segments=bound)
        n = lg.grouped_workspace_bytes(rows, slots, sum(s[0] for s in shapes.values()), len(shapes))
        self.ws = torch.full((max(n, 16),), 0x7f, dtype=torch.uint8, device="cuda")
        self.dids = torch.from_numpy(self.ids).cuda()
        self.upload()

    def upload(self):
        self.table = torch.from_numpy(self.host.view(np.uint8).reshape(-1).copy()).cuda()

    def launch(self):
        lg.build_segments(self.dids, self.slots, self.seg, self.ws)
        lg.grouped_layer(self.dev, self.rows, self.table, self.slots, self.seg, self.ws, int8=self.int8)

    def out(self):
        return {m: io.y.clone() for m, io in self.dev.items()}

    def run(self):
        for io in self.dev.values():
            io.y.fill_(7.0)
        self.launch()
        torch.cuda.synchronize()
        return self.out()

    def check(self, got=None, skip=()):
        got = self.run() if got is None else got
        for m, (di, do, _) in self.shapes.items():
            c = self.cpu[m]
            done = np.zeros(self.rows, bool)
            for s in range(self.slots):
                at = np.nonzero(self.ids == s)[0]
                if len(at) == 0 or s in self.none or s in skip:
                    continue
                done[at] = True
                x = c["x"][at // self.fan]
                ref, slack = base_i8(x, c["W"][s], c["Ws"][s]) if self.int8 else grouped_bf16(x, c["W"][s])
                close(got[m][torch.from_numpy(at).cuda()][:, :do], ref, slack, f"{m} slot {s}")
            rest = torch.from_numpy(np.nonzero(~done)[0]).cuda()
            assert bool((got[m][rest] == 7).all()), f"{m}: rows without a weight were written"
            assert bool((got[m][:, do:] == 7).all()), f"{m}: columns past d_out were written"


def ragged(lengths, seed=0, shuffle=True):
    ids = np.repeat(np.arange(len(lengths)), lengths)
    if shuffle:
        ids = np.random.RandomState(seed).permutation(ids)
    return ids


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("rows,slots", [(1, 1), (2, 9), (16, 4), (17, 1), (40, 3), (65, 2), (130, 1), (260, 3), (700, 2),
                                        (300, 150)])
def test_rows(int8, rows, slots):
    Run(int8, ids_of("mixed", rows, slots, rows), slots, {"q": (264, 136, "a"), "k": (264, 72, "a")}, seed=rows).check()


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("lengths", [(0, 1, 0, 16, 17), (1,) * 70, (128, 0, 129, 1), (255, 257, 3, 64), (0, 0, 0, 5),
                                     (1000, 1, 1, 1), (16, 32, 64, 128)])
@pytest.mark.parametrize("shuffle", [False, True])
def test_ragged(int8, lengths, shuffle):
    Run(int8, ragged(lengths, 1, shuffle), len(lengths), {"o": (136, 200, "o")}, seed=len(lengths)).check()


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("d_in,d_out", [(8, 8), (24, 16), (56, 8), (64, 128), (72, 136), (120, 24), (256, 32), (264, 40),
                                        (520, 264), (1032, 72), (4104, 16)])
@pytest.mark.parametrize("rows", [3, 50, 120, 400])
def test_widths(int8, d_in, d_out, rows):
    Run(int8, ids_of("mixed", rows, 2, d_in), 2, {"down": (d_in, d_out, "d")}, seed=d_in + d_out).check()


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("fan,rows", [(2, 64), (3, 100), (8, 33), (5, 1), (2, 600)])
def test_rows_that_share_x(int8, fan, rows):
    Run(int8, ids_of("mixed", rows, 6, fan), 6, {"gate": (264, 200, "m"), "up": (264, 200, "m")}, fan=fan, seed=fan).check()


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("lengths", [(1300, 900, 1901), (4100,)])
def test_largest_tile(int8, lengths):
    # at least 256 tiles of 256 x 256, partial ones at both edges
    Run(int8, ragged(lengths, 3), len(lengths), {"q": (136, 5128, "a")}, seed=7).check()


@pytest.mark.parametrize("int8", FORMS)
def test_many_segments(int8):
    # more segments than a wave looks at in one step, at a small and at a large row tile
    Run(int8, ids_of("mixed", 900, 300, 5), 300, {"k": (72, 40, "a")}, seed=9).check()
    Run(int8, ragged([65 + (i * 37) % 90 for i in range(140)], 2), 140, {"k": (40, 24, "a")}, seed=10).check()


@pytest.mark.parametrize("int8", FORMS)
def test_strided(int8):
    Run(int8, ids_of("mixed", 45, 4, 1), 4, {"q": (264, 136, "a"), "o": (136, 264, "o")}, seed=4, pad=16).check()


@pytest.mark.parametrize("int8", FORMS)
def test_slots_without_a_weight(int8):
    r = Run(int8, ids_of("mixed", 60, 5, 1), 5, {"q": (136, 72, "a")}, seed=5, none=(1, 3))
    r.check()
    assert int(r.seg.status.item()) == int((r.ids >= 5).sum())


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("rows", [60, 400])
def test_bad_entries_count_once_and_skip(int8, rows):
    r = Run(int8, ids_of("mixed", rows, 6, 2), 6, {"q": (136, 264, "a"), "o": (136, 72, "o")}, seed=6)
    r.host["W"][1, 0] += 8
    r.host["ldw"][2, 0] = 128          # below d_in
    r.host["ldw"][3, 0] += 4           # rows not 16-byte aligned
    r.host["ldw"][5, 0] = 1 << 33      # past 4 GiB
    if int8:
        r.host["Ws"][4, 0] = 0
    r.upload()
    skip = (1, 2, 3, 5) + ((4,) if int8 else ())
    got = r.run()
    assert int(r.seg.status.item()) == int((r.ids >= 6).sum()) + sum(s in set(r.ids.tolist()) for s in skip)
    shapes = dict(r.shapes)
    r.shapes = {"q": shapes["q"]}
    r.check(got, skip)
    r.shapes = {"o": shapes["o"]}
    r.check(got)


@pytest.mark.parametrize("int8", FORMS)
def test_segments_of_another_batch_are_skipped(int8):
    # segments built for more rows than the call's batch: those that reach past it are counted, the rest applied
    r = Run(int8, ragged([10, 10, 10], shuffle=False), 3, {"q": (136, 72, "a")}, seed=12)
    for io in r.dev.values():
        io.y.fill_(7.0)
    lg.build_segments(r.dids, r.slots, r.seg, r.ws)
    lg.grouped_layer(r.dev, 25, r.table, r.slots, r.seg, r.ws, int8=int8)
    torch.cuda.synchronize()
    assert int(r.seg.status.item()) == 1
    r.check(r.out(), skip=(2,))


@pytest.mark.parametrize("int8", FORMS)
def test_segment_bound(int8):
    r = Run(int8, ids_of("mixed", 80, 40, 3), 40, {"q": (136, 72, "a")}, seed=13, bound=7)
    r.check(skip=sorted(set(i for i in r.ids.tolist() if 0 <= i < 40))[7:])


@pytest.mark.parametrize("int8", FORMS)
def test_non_finite_rows_and_weights_stay_alone(int8):
    r = Run(int8, ids_of("mixed", 50, 4, 4), 4, {"q": (264, 72, "a")}, seed=14)
    x = r.cpu["q"]["x"].clone()
    x[7, 100] = float("nan")
    r.cpu["q"]["x"] = x
    r.dev["q"].x.copy_(x)
    clean = torch.ones(50, dtype=torch.bool)
    clean[7] = False
    if not int8:
        r.keep["q", 2][0][11, 5] = float("inf")
    got = r.run()["q"].cpu()
    for s in range(4):
        at = np.nonzero((r.ids == s) & clean.numpy())[0]
        ref, slack = (base_i8(x[at], r.cpu["q"]["W"][s], r.cpu["q"]["Ws"][s]) if int8
                      else grouped_bf16(x[at], r.cpu["q"]["W"][s]))
        cols = np.arange(72) != (11 if s == 2 and not int8 else -1)
        close(got[at][:, cols], ref[:, cols], slack[:, cols], f"slot {s}")
    if 0 <= r.ids[7] < 4:
        assert bool(torch.isnan(got[7]).all())


@pytest.mark.parametrize("rows,fan", [(1, 1), (37, 2), (300, 1)])
def test_workspace_is_not_overrun(rows, fan):
    shapes = {"q": (1032, 72, "a"), "o": (8, 264, "o"), "down": (4104, 16, "d")}
    r = Run(True, ids_of("mixed", rows, 5, 2), 5, shapes, fan=fan, seed=17)
    n = lg.grouped_workspace_bytes(rows, 5, sum(s[0] for s in shapes.values()), len(shapes))
    big = torch.full((n + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    r.ws = big[:n]
    r.check()
    assert bool((big[n:] == 0x5a).all())


@pytest.mark.parametrize("int8", FORMS)
def test_no_rows(int8):
    r = Run(int8, [-1] * 20, 3, {"q": (136, 72, "a")}, seed=15)
    r.check()
    r.rows = 0
    lg.grouped_layer(r.dev, 0, r.table, r.slots, r.seg, r.ws, int8=int8)
    torch.cuda.synchronize()
    assert bool((r.out()["q"] == 7).all())


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("rows", [5, 90, 400])
def test_graph_replays(int8, rows):
    r = Run(int8, ids_of("mixed", rows, 6, 1), 6, {"q": (264, 136, "a"), "k": (264, 72, "a")}, seed=16)
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
            io.y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got, eager = r.out(), r.run()
        for m in got:
            assert torch.equal(got[m], want[m]) and torch.equal(eager[m], want[m]), (k, m)
    r.ids = ids_of("runs", rows, 6, 8)
    r.dids.copy_(torch.from_numpy(r.ids))
    for io in r.dev.values():
        io.y.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    r.check(r.out())


def test_merged_rows_beside_low_rank_rows():
    """A batch whose slots 0..2 are merged weights and 3..5 low-rank adapters
    on an int8 base: one build of the segments serves both calls, each writes
    its own rows."""
    from tests.test_gpu_linear_i8 import Run as Linear
    rows, slots = 60, 6
    lin = Linear(rows, slots, {"q": (264, 136, "a")}, (16, 8), "mixed", seed=71)
    lin.table_host["rank"][:3, 0] = 0
    lin.upload()
    grp = Run(False, lin.ids, slots, {"q": (264, 136, "a")}, seed=72, none=(3, 4, 5))
    lin.launch()
    y = lin.dev["q"].y
    ios = {"q": lg.GroupedIO(lin.dev["q"].x, y)}
    lg.grouped_layer(ios, rows, grp.table, slots, lin.seg)
    torch.cuda.synchronize()
    ref, slack = lin.reference("q", skip=(0, 1, 2))
    for s in range(3):
        at = np.nonzero(lin.ids == s)[0]
        ref[at], slack[at] = grouped_bf16(lin.cpu["q"]["x"][at], grp.cpu["q"]["W"][s])
    close(y, ref, slack, "mixed batch")


@pytest.mark.parametrize("int8", FORMS)
def test_experts_of_an_mlp(int8):
    """gate, up, silu, down through two of eight experts per token, as a
    mixture-of-experts layer runs them."""
    tokens, fan, slots, d, ffn = 40, 2, 8, 264, 200
    r = np.random.RandomState(5)
    ids = np.concatenate([r.permutation(slots)[:fan] for _ in range(tokens)])
    up = Run(int8, ids, slots, {"gate": (d, ffn, "m"), "up": (d, ffn, "m")}, fan=fan, seed=81)
    got = up.run()
    up.check(got)
    h = (torch.nn.functional.silu(got["gate"].float()) * got["up"].float()).to(torch.bfloat16)
    down = Run(int8, ids, slots, {"down": (ffn, d, "d")}, seed=82)
    down.dev["down"].x = h
    down.cpu["down"]["x"] = h.cpu()
    down.check()


@pytest.mark.parametrize("int8", FORMS)
def test_offsets_near_4_gib(int8):
    """x rows and weight rows so far apart that the last ones start just below 4 GiB."""
    rows, d = 262000, 72
    ldx = 8192 - 8                                   # 262000 rows * 16368 bytes
    r = Run(int8, ids_of("mixed", 300, 2, 3), 2, {"q": (d, 40, "a")}, seed=91)
    keep = [0, 1, rows // 2, rows - 2, rows - 1]
    ids = np.full(rows, -1, np.int32)
    ids[keep] = [0, 1, 1, 0, 1]
    x = torch.zeros(rows * ldx, dtype=torch.bfloat16, device="cuda").view(rows, ldx)
    xs = bf16(gen(5), len(keep), d)
    x[keep, :d] = xs.cuda()
    y = torch.full((rows, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    elt = 1 if int8 else 2
    ldw = (4294967040 // elt // 40) // 16 * 16
    host = r.host.copy()
    big = torch.zeros(40 * ldw, dtype=torch.int8 if int8 else torch.bfloat16, device="cuda").view(40, ldw)
    W = r.cpu["q"]["W"][1]
    big[:, :d] = W.cuda()
    host["W"][1, 0], host["ldw"][1, 0] = big.data_ptr(), ldw
    table = torch.from_numpy(host.view(np.uint8).reshape(-1).copy()).cuda()
    seg = lg.Segments(rows, max_segments=2)
    ws = torch.empty(max(lg.grouped_workspace_bytes(rows, 2, d, 1), 16), dtype=torch.uint8, device="cuda")
    dids = torch.from_numpy(ids).cuda()
    lg.build_segments(dids, 2, seg, ws)
    lg.grouped_layer({"q": lg.GroupedIO(x, y, d_in=d)}, rows, table, 2, seg, ws, int8=int8)
    torch.cuda.synchronize()
    assert int(seg.status.item()) == 0
    for i, b in enumerate(keep):
        a = int(ids[b])
        Ws = r.cpu["q"]["Ws"][a]
        ref, slack = (base_i8(xs[i:i + 1], r.cpu["q"]["W"][a], Ws) if int8 else grouped_bf16(xs[i:i + 1], r.cpu["q"]["W"][a]))
        close(y[b:b + 1], ref, slack, f"row {b}")
    y[keep] = 7.0
    assert bool((y == 7).all())


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("lengths,rows", [((10, 10, 10), 25), ((10, 10, 10), 21), ((5, 1, 40, 9, 30), 60), ((70, 60, 90), 150),
                                          ((300, 280, 520), 700)])
def test_rows_past_the_batch_in_segments_that_fit_touch_nothing(int8, lengths, rows):
    stray_rows(int8, lengths, rows, {"q": (136, 200, "a"), "o": (72, 40, "o")})


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("tile,lengths,rows,d_out", [((128, 128), (127, 4, 129), 200, 8200), ((256, 256), (300, 200, 260), 560, 12296)])
def test_rows_past_the_batch_touch_nothing_on_tiles_that_store_whole_lines(int8, tile, lengths, rows, d_out):
    assert tile_of("grouped_i8" if int8 else "grouped", rows, len(lengths), [(136, d_out)]) == tile
    stray_rows(int8, lengths, rows, {"q": (136, d_out, "a")})


def stray_rows(int8, lengths, rows, shapes):
    # segments of a longer, shuffled batch: those that end inside this one hold rows past it, which are skipped; no row of
    # this batch gets another row's result, the last one (and rows past it) included
    r = Run(int8, ragged(lengths, 4), len(lengths), shapes, seed=19)
    fit = [s for s in range(len(lengths)) if sum(lengths[:s + 1]) <= rows]
    assert any((r.ids[rows:] == s).any() for s in fit)  # stray rows are there
    for io in r.dev.values():
        io.y.fill_(7.0)
    lg.build_segments(r.dids, r.slots, r.seg, r.ws)
    lg.grouped_layer(r.dev, rows, r.table, r.slots, r.seg, r.ws, int8=int8)
    torch.cuda.synchronize()
    assert int(r.seg.status.item()) == len(lengths) - len(fit)
    got = r.out()
    for m in got:
        assert bool((got[m][rows:] == 7).all()), m
    r.ids = np.where(np.arange(r.rows) < rows, r.ids, -1)
    r.check(got, skip=[s for s in range(len(lengths)) if s not in fit])


def test_rows_and_scales_at_the_ends_of_the_type():
    # int8: the row scale and the output scale multiply a sum of 2^23 without leaving the type on the way (four
    # roundings); every row once under each of two slots
    d = 264
    ids = np.arange(24) % 2
    r = Run(True, ids, 2, {"q": (d, 64, "a")}, fan=2, seed=18)
    x = extreme_rows(d)
    r.dev["q"].x.copy_(x)
    for s in (0, 1):
        r.cpu["q"]["Ws"][s] = extreme_scales(r.cpu["q"]["Ws"][s])
        r.keep["q", s][1].copy_(r.cpu["q"]["Ws"][s])
    got = r.run()["q"]
    for s in (0, 1):
        ref, _ = base_i8(x, r.cpu["q"]["W"][s], r.cpu["q"]["Ws"][s])
        close_range(got[s::2], ref, 4 * U, f"slot {s}")


@pytest.mark.parametrize("int8", FORMS)
@pytest.mark.parametrize("tile,lengths,d_in,d_out", GROUPED_TILES)
def test_each_tile(int8, tile, lengths, d_in, d_out):
    # every kernel, its ring filled again and its edges partial
    assert tile_of("grouped_i8" if int8 else "grouped", sum(lengths), len(lengths), [(d_in, d_out)]) == tile
    Run(int8, ragged(lengths, 5), len(lengths), {"q": (d_in, d_out, "a")}, seed=len(lengths) + d_in).check()
