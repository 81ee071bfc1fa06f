"""GPU tests of the calls with one base weight and the rows' adapters that are
4-bit in stated groups or gated (lora_linear_layer_q4g, lora_gated_layer,
lora_gated_layer_q4g) against the 64-bit definition."""
import numpy as np
import pytest

from tests.dense_cases import MODS, bf16, close, delta, gen, grouped_bf16, ids_of
from tests.ffn_cases import ACTS, GROUPS, TILE_SLOTS, TILES, gated, q4_sums, q4_weight
from tests.parity import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import adapter_gemv_amd as lg  # noqa: E402

# (gated, group): group 0 is bf16
FORMS = [(False, 128), (False, 32), (True, 0), (True, 128), (True, 32)]
IDS = ["q4g128", "q4g32", "gated", "gated-q4g128", "gated-q4g32"]
forms = pytest.mark.parametrize("form", FORMS, ids=IDS)


@pytest.fixture(autouse=True)
def _name_case(request):
    note(request.node.nodeid)


def fit(d_in, group):
    return d_in if group == 0 else max(group, -(-d_in // group) * group)


def int8_factors(A, B):
    """(A fp64, B fp64, A block, B block) of LORA_FORMAT_INT8_ROWS."""
    def q(t):
        t = t.float()
        s = t.abs().amax(1) / 127 + 1e-6
        return torch.round(t / s[:, None]).clamp(-127, 127).to(torch.int8), s

    def block(qv, s, ld):
        sc = torch.zeros(-(-s.numel() // 4) * 4)
        sc[:s.numel()] = s
        v = torch.zeros(qv.shape[0], ld, dtype=torch.int8)
        v[:, :qv.shape[1]] = qv
        return torch.cat([sc.view(torch.uint8), v.view(torch.uint8).reshape(-1)]).cuda()

    qa, sa = q(A)
    qb, sb = q(B)
    return (qa.double() * sa.double()[:, None], qb.double() * sb.double()[:, None],
            block(qa, sa, -(-A.shape[1] // 16) * 16), block(qb, sb, -(-max(B.shape[1], 1) // 16) * 16))


class Run:
    """A batch with adapters.  shapes: {projection: (d_in, d_out, what its x is called)}; gated: "gate" stands for both."""

    def __init__(self, form, rows, slots, shapes, ranks, kind="mixed", seed=0, fmt="bf16", pad=0, bound=0, act="silu",
                 x_std=1.0):
        g = gen(seed + 1)
        self.is_gated, self.group = form
        self.rows, self.slots, self.act = rows, slots, act
        self.shapes = {m: (fit(s[0], self.group),) + s[1:] for m, s in shapes.items()}
        self.ids = ids_of(kind, rows, slots, seed)
        ranks = [ranks] * slots if isinstance(ranks, int) else [ranks[s % len(ranks)] for s in range(slots)]
        self.max_rank = max(max(ranks), 1)
        self.cpu, self.dev, self.keep = {}, {}, []
        shape = (slots, 7)
        A_p, B_p, rk = np.zeros(shape, np.uint64), np.zeros(shape, np.uint64), np.zeros(shape, np.int32)
        sc, fm = np.ones(shape, np.float32), np.zeros(shape, np.int32)
        xs = {}
        for m, (di, do, share) in self.shapes.items():
            if share not in xs:
                full = bf16(g, max(rows, 1), di + pad, std=x_std)
                xs[share] = (full, full.cuda())
            y = torch.full((max(rows, 1), do + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
            weights = []
            for col in ("gate", "up") if self.is_gated else (m,):
                c = {"x": xs[share][0][:, :di], "A": [], "B": [], "scale": []}
                if self.group:
                    Wq, Ws, W = q4_weight(g, do, di, self.group, 2 * pad, pad // 8)
                    c["W"] = (W, Ws, self.group)
                    weights += [Wq.cuda(), Ws.cuda()]
                else:
                    full = bf16(g, do, di + pad, std=di ** -0.5)
                    c["W"] = (full[:, :di],)
                    weights.append(full.cuda())
                k = MODS.index(col)
                for s in range(slots):
                    r = ranks[(s + k) % len(ranks)] if self.is_gated else ranks[s]
                    A, B = bf16(g, r, di, std=0.1), bf16(g, do, r, std=0.1)
                    scale = float(np.float32(0.25 + 0.5 * ((s * 7 + k) % 5)))
                    if r and (fmt == "int8" or (fmt == "both" and s % 2)):
                        A, B, pa, pb = int8_factors(A, B)
                        fm[s, k] = lg.FORMAT_INT8_ROWS
                    else:
                        Bp = torch.zeros(do, -(-max(r, 1) // 8) * 8, dtype=torch.bfloat16)
                        Bp[:, :r] = B
                        pa, pb = A.cuda(), Bp.cuda()
                    self.keep += [pa, pb]
                    A_p[s, k], B_p[s, k] = (pa.data_ptr(), pb.data_ptr()) if r else (0, 0)
                    rk[s, k], sc[s, k] = r, scale
                    c["A"].append(A)
                    c["B"].append(B)
                    c["scale"].append(scale)
                self.cpu[col] = c
            x = xs[share][1]
            if not self.is_gated:
                self.dev[m] = lg.LinearQ4GIO(x, *weights, y, self.group, d_in=di, d_out=do)
            elif self.group:
                self.dev[m] = lg.GatedQ4GIO(x, *weights, y, self.group, d_in=di, d_ff=do)
            else:
                self.dev[m] = lg.GatedIO(x, *weights, y, d_in=di, d_ff=do)
        self.table_host = lg.pack_table(A_p, B_p, rk, sc, fm)
        self.seg = lg.Segments(rows, max_segments=bound)
        if self.is_gated:
            n = lg.gated_workspace_bytes(rows, slots, self.max_rank, self.shapes["gate"][0])
        else:
            n = lg.linear_q4g_workspace_bytes(rows, slots, self.max_rank, sum(s[0] for s in self.shapes.values()),
                                              len(self.shapes))
        self.ws = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
        self.dids = torch.from_numpy(self.ids).cuda()
        self.upload()

    def upload(self):
        self.table = torch.from_numpy(self.table_host.view(np.uint8).reshape(-1).copy()).cuda()

    def call(self, rows=None, stream=None):
        rows = self.rows if rows is None else rows
        if self.is_gated:
            lg.gated_layer(self.dev["gate"], rows, self.dids, self.table, self.slots, self.seg, self.max_rank, self.ws,
                           stream=stream, activation=self.act)
        else:
            lg.linear_layer(self.dev, rows, self.dids, self.table, self.slots, self.seg, self.max_rank, self.ws,
                            stream=stream)

    def launch(self, stream=None):
        lg.build_segments(self.dids, self.slots, self.seg, self.ws, stream=stream)
        self.call(stream=stream)

    def out(self, m):
        return self.dev[m].h if self.is_gated else self.dev[m].y

    def run(self):
        for m in self.dev:
            self.out(m).fill_(float("nan"))
        self.launch()
        torch.cuda.synchronize()
        return {m: self.out(m).clone() for m in self.dev}

    def status(self):
        return int(self.seg.status.item())

    def sums(self, col, skip=()):
        """(projection, slack) in fp64; skip: slots that get no delta."""
        c = self.cpu[col]
        y, slack = (q4_sums if self.group else grouped_bf16)(c["x"][:self.rows], *c["W"])
        for s in range(self.slots):
            at = np.nonzero(self.ids == s)[0]
            if len(at) and s not in skip and c["A"][s].shape[0]:
                d, sl = delta(c["x"][at], c["A"][s], c["B"][s], c["scale"][s])
                y[at] += d
                slack[at] += sl
        return y, slack

    def check(self, got=None, skip=()):
        got = self.run() if got is None else got
        for m, (di, do, _) in self.shapes.items():
            if self.is_gated:
                ref, slack = gated(self.act, *self.sums("gate", skip), *self.sums("up", skip))
            else:
                ref, slack = self.sums(m, skip)
            close(got[m][:self.rows, :do], ref, slack, m)
            assert bool(torch.isnan(got[m][:, do:]).all()), f"{m}: columns past the output were written"


def one(d_in, d_out):
    return {"gate": (d_in, d_out, "m")}


@forms
@pytest.mark.parametrize("rows,slots", [(1, 1), (2, 9), (16, 4), (17, 1), (40, 3), (63, 7), (64, 5), (65, 2), (130, 1),
                                        (260, 3), (700, 9), (300, 150)])
def test_rows(form, rows, slots):
    Run(form, rows, slots, one(264, 136), [5, 16, 0, 32], seed=rows).check()


@pytest.mark.parametrize("group,rank", [(32, 48), (128, 16)])
@pytest.mark.parametrize("kind,number,tile,rows,d_in,d_out", [c for c in TILES if not c[0].startswith("grouped")])
def test_every_tile(kind, number, tile, rows, d_in, d_out, group, rank):
    if not kind.endswith("q4g"):
        group = 0
    Run(("gated" in kind, group), rows, TILE_SLOTS, one(d_in, d_out), rank, seed=tile[0], fmt="both").check()


@forms
@pytest.mark.parametrize("rows,rank", [(15, 64), (48, 16), (63, 64), (64, 16)])
def test_either_way_to_v(form, rows, rank):
    # few rows without the grouped shrink, and the same sizes past its bound of work or rows
    # (the 63 rows with the longer d_in: past 192 MB of factors and x)
    Run(form, rows, 20, one(4104 if form[1] == 0 else 4096, 72), rank, seed=rows, fmt="both").check()
    if rows == 63:
        Run(form, rows, 20, one(16384, 40), rank, seed=rows, fmt="both").check()


@pytest.mark.parametrize("is_gated,group", [(False, 32), (False, 64), (False, 128), (True, 0), (True, 32), (True, 128)])
@pytest.mark.parametrize("rows", [1, 4, 16])
def test_few_rows_over_a_long_input(is_gated, group, rows):
    # blocks start at different places along k and come round; many batches of scales
    Run((is_gated, group), rows, 3, one(8192 + (group or 8), 2056), 16, seed=rows).check()


@forms
@pytest.mark.parametrize("rank", [1, 7, 8, 16, 31, 32, 33, 48, 64])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "both"])
@pytest.mark.parametrize("rows", [6, 100, 300])
def test_ranks_and_formats(form, rank, fmt, rows):
    Run(form, rows, 5, one(264, 136), rank, fmt=fmt, seed=rank, act="gelu_tanh").check()


@forms
@pytest.mark.parametrize("kind", ["distinct", "runs", "one", "none", "mixed"])
@pytest.mark.parametrize("rows", [20, 150, 600])
def test_batches(form, kind, rows):
    Run(form, rows, 40, one(264, 200), [16, 8], kind=kind, seed=3).check()


@forms
@pytest.mark.parametrize("d_in,d_out", [(8, 8), (24, 16), (64, 128), (72, 136), (120, 24), (520, 264), (1032, 72), (4104, 16)])
@pytest.mark.parametrize("rows", [3, 50, 120, 400])
def test_widths(form, d_in, d_out, rows):
    Run(form, rows, 3, one(d_in, d_out), [16, 5], seed=d_in + d_out).check()


@pytest.mark.parametrize("is_gated", [False, True])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("groups", [1, 2, 3, 5, 9, 17])
@pytest.mark.parametrize("rows", [1, 100, 300])
def test_groups(is_gated, group, groups, rows):
    Run((is_gated, group), rows, 2, one(group * groups, 72), 8, seed=groups).check()


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("rows", [1, 33, 300])
def test_all_projections(group, rows):
    shapes = {"q": (256, 136, "a"), "k": (256, 40, "a"), "v": (256, 40, "a"), "o": (384, 256, "o"), "gate": (256, 520, "m"),
              "up": (256, 520, "m"), "down": (640, 256, "d")}
    Run((False, group), rows, 6, shapes, [16, 32, 8], seed=rows, pad=8).check()


@forms
@pytest.mark.parametrize("pad", [8, 24])
def test_strides(form, pad):
    for rows in (9, 200):
        Run(form, rows, 3, one(264, 136), 16, pad=pad, seed=pad).check()


@forms
@pytest.mark.parametrize("rows", [12, 90])
@pytest.mark.parametrize("bound", [2, 4])
def test_a_bound_on_the_segments(form, rows, bound):
    r = Run(form, rows, 4, one(264, 136), 16, seed=9, bound=bound)
    kept = np.unique(r.ids[(r.ids >= 0) & (r.ids < 4)])[:bound]
    r.check(skip=[s for s in range(4) if s not in kept])


@forms
@pytest.mark.parametrize("rows", [60, 90])
def test_bad_entries_are_counted_and_get_no_delta(form, rows):
    r = Run(form, rows, 5, one(264, 136), 16, kind="runs", seed=4)
    cols = [MODS.index(c) for c in (("gate", "up") if r.is_gated else ("gate",))]
    present = [s for s in range(5) if (r.ids == s).any()]
    for k in cols:
        r.table_host["rank"][0, k] = 17
        r.table_host["B"][1, k] += 8
        r.table_host["A"][2, k] = 0
        r.table_host["format"][3, k] = 9
    r.upload()
    r.check(skip=[0, 1, 2, 3])
    assert r.status() == len(cols) * len([s for s in present if s < 4])


def test_one_projection_of_a_slot_without_adapter():
    # rank 0 in one column, a bad entry in the other: each has its own delta or none
    r = Run((True, 0), 40, 3, one(264, 136), 16, seed=4)
    up = MODS.index("up")
    r.table_host["rank"][0, up] = 0
    r.table_host["B"][1, up] = 0
    r.upload()
    got = r.run()
    ref, slack = gated(r.act, *r.sums("gate"), *r.sums("up", skip=[0, 1]))
    close(got["gate"][:, :136], ref, slack, "gate")
    assert r.status() == int((r.ids >= 3).sum()) + int((r.ids == 1).any())


@forms
def test_another_tenants_broken_factors_reach_no_other_row(form):
    r = Run(form, 70, 4, one(264, 136), 16, seed=2)
    clean = r.run()["gate"].clone()
    for t in r.keep[2:4]:  # slot 1 of the first projection
        t.fill_(float("nan"))
    got = r.run()["gate"]
    keep = torch.from_numpy(np.nonzero(r.ids != 1)[0]).cuda()
    assert torch.equal(got[keep, :136], clean[keep, :136])
    assert bool(torch.isnan(got[torch.from_numpy(r.ids == 1).cuda()][:, :136]).all())


@forms
def test_a_row_with_nan_or_infinity_reaches_no_other(form):
    r = Run(form, 70, 3, one(264, 136), 16, seed=6)
    clean = r.run()["gate"].clone()
    x = r.dev["gate"].x
    x[5, 7], x[11, :], x[39, 0], x[66, 3] = float("nan"), float("inf"), float("-inf"), float("nan")
    got = r.run()["gate"]
    keep = torch.tensor([i for i in range(70) if i not in (5, 11, 39, 66)], device="cuda")
    assert torch.equal(got[keep, :136], clean[keep, :136])
    assert bool(torch.isnan(got[5, :136]).all()) and bool(torch.isnan(got[66, :136]).all())


@forms
@pytest.mark.parametrize("rows", [12, 300])
def test_captured_and_replayed(form, rows):
    r = Run(form, rows, 4, one(520, 136), 16, seed=rows)
    want = r.run()["gate"].clone()
    assert torch.equal(r.run()["gate"][:, :136], want[:, :136])  # bits repeat
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.launch()
    for k in range(3):
        r.out("gate").fill_(float("nan"))
        r.ws.fill_(0x7f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.out("gate")[:, :136], want[:, :136]), f"replay {k}"
    r.ids = r.ids[::-1].copy()  # other ids and factors, read at the replay
    r.dids.copy_(torch.from_numpy(r.ids))
    r.table_host["scale"][:] *= 2
    for c in r.cpu.values():
        c["scale"] = [2 * s for s in c["scale"]]
    r.table.copy_(torch.from_numpy(r.table_host.view(np.uint8).reshape(-1).copy()))
    r.out("gate").fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    r.check({"gate": r.out("gate")})


@forms
def test_two_streams_at_once(form):
    runs = [Run(form, 130, 4, one(1032, 264), 16, seed=k) for k in range(2)]
    want = [r.run()["gate"].clone() for r in runs]
    sides = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(4):
        for r, s in zip(runs, sides):
            r.launch(stream=s)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert torch.equal(r.out("gate")[:, :264], w[:, :264])


@forms
def test_no_rows(form):
    r = Run(form, 0, 2, one(264, 136), 16)
    r.run()
    assert bool(torch.isnan(r.out("gate")).all())


@forms
@pytest.mark.parametrize("rows,fewer", [(100, 70), (100, 40)])
def test_segments_of_a_longer_batch(form, rows, fewer):
    # a call for fewer rows than the segments hold: no delta for a segment that does not fit, which is counted, and
    # nothing past the rows
    r = Run(form, rows, 3, one(264, 136), 16, kind="one", seed=5)
    r.ids = np.sort(np.random.RandomState(3).randint(0, 3, rows)).astype(np.int32)
    r.dids.copy_(torch.from_numpy(r.ids))
    lg.build_segments(r.dids, 3, r.seg, r.ws)
    r.out("gate").fill_(float("nan"))
    r.call(rows=fewer)
    torch.cuda.synchronize()
    assert bool(torch.isnan(r.out("gate")[fewer:]).all())
    ends = np.cumsum(np.bincount(r.ids, minlength=3))
    out = [s for s in range(3) if ends[s] > fewer]
    assert 0 < len(out) < 3
    # 64 rows and more: counted by the grouped shrink, a segment of 8 rows and more by both of its parts
    assert r.status() == len(out) if fewer < 64 else len(out) <= r.status() <= 2 * len(out)
    r.rows, full = fewer, r.ids
    r.ids = full[:fewer]
    r.check({"gate": r.out("gate")}, skip=out)


@forms
@pytest.mark.parametrize("rows,kept", [(90, 37), (600, 300)])
def test_ids_other_than_the_segments(form, rows, kept):
    # rows that get a slot after the segments were built are in no segment and not among the rows without one: they
    # may be left unwritten, and the others keep their results
    r = Run(form, rows, 3, one(264, 136), 16, seed=5)
    r.ids = np.sort(np.random.RandomState(3).randint(0, 3, rows)).astype(np.int32)
    r.ids[kept:] = -1
    r.dids.copy_(torch.from_numpy(r.ids))
    lg.build_segments(r.dids, 3, r.seg, r.ws)
    r.dids[kept:] = 0
    r.ws.fill_(0x7f)
    r.out("gate").fill_(float("nan"))
    r.call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(r.out("gate")[kept:]).all())
    assert r.status() == 0
    r.rows, r.ids = kept, r.ids[:kept]
    r.check({"gate": r.out("gate")})


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("act", ACTS)
def test_activation_over_its_range(group, act):
    for std in (2.0 ** -60, 0.1, 30.0, 3000.0):
        Run((True, group), 60, 2, one(264, 136), 16, act=act, x_std=std, seed=int(std)).check()


def test_a_layers_block_together():
    """The gated half and the down projection of a 4-bit base with the same rows' adapters, as one captured decode step."""
    d, f, group, rows = 256, 640, 64, 24
    a = Run((True, group), rows, 5, one(d, f), 16, seed=1)
    b = Run((False, group), rows, 5, {"down": (f, d, "h")}, 16, seed=1)
    b.dev["down"].x = a.out("gate")

    def step():
        a.launch()
        lg.linear_layer(b.dev, rows, a.dids, b.table, 5, a.seg, 16, b.ws)

    step()
    torch.cuda.synchronize()
    a.check({"gate": a.out("gate").clone()})
    b.cpu["down"]["x"] = a.out("gate").cpu()
    want = b.out("down").clone()
    b.check({"down": want})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        a.out("gate").fill_(float("nan"))
        b.out("down").fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out("down"), want)
