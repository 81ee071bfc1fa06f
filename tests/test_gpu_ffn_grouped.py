"""GPU tests of the products with a weight per slot that are 4-bit or gated
(lora_grouped_layer_q4g, lora_grouped_gated_layer, lora_grouped_gated_layer_q4g)
against the 64-bit definition."""
import numpy as np
import pytest

from tests.dense_cases import MODS, bf16, close, gen, grouped_bf16, ids_of
from tests.ffn_cases import ACTS, GROUPS, TILES, gated, q4_sums, q4_weight
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
    """The nearest width that the group divides."""
    return d_in if group == 0 else max(group, -(-d_in // group) * group)


class Run:
    """A batch with a weight per slot.  shapes: {projection: (d_in, d_out, what its x is called)}; gated: of "gate" alone."""

    def __init__(self, form, ids, slots, shapes, fan=1, seed=0, pad=0, bound=0, none=(), act="silu", x_std=1.0):
        g = gen(seed + 1)
        self.is_gated, self.group = form
        self.ids, self.slots, self.fan, self.act = np.asarray(ids, np.int32), slots, fan, act
        self.shapes = {m: (fit(s[0], self.group),) + s[1:] for m, s in shapes.items()}
        self.rows = rows = len(ids)
        self.none = set(none)
        self.cpu, self.dev, self.keep = {}, {}, []
        t = np.zeros((slots, 7), lg.WEIGHT_Q4G_ENTRY_DTYPE)
        xs = {}
        for m, (di, do, share) in self.shapes.items():
            if share not in xs:
                full = bf16(g, max(-(-rows // fan), 1), di + pad, std=x_std)
                xs[share] = (full, full.cuda())
            y = torch.full((max(rows, 1), do + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            self.dev[m] = lg.GroupedIO(xs[share][1], y, d_in=di, d_out=do, rows_per_x=fan)
            self.cpu[m] = {"x": xs[share][0][:, :di], "W": {}}
            for col in ("gate", "up") if self.is_gated else (m,):
                for s in range(slots):
                    if self.group:
                        Wq, Ws, W = q4_weight(g, do, di, self.group, 2 * pad, pad // 8)
                        dw, ds = Wq.cuda(), Ws.cuda()
                    else:
                        full = bf16(g, do, di + pad, std=di ** -0.5)
                        W, dw, ds = full[:, :di], full.cuda(), None
                    self.keep.append((dw, ds))
                    self.cpu[m]["W"][col, s] = (W, Ws, self.group) if self.group else (W,)
                    if s not in self.none:
                        c = MODS.index(col)
                        t["W"][s, c], t["ldw"][s, c] = dw.data_ptr(), dw.stride(0)
                        if ds is not None:
                            t["Ws"][s, c], t["lds"][s, c] = ds.data_ptr(), ds.stride(0)
        self.host = t
        self.seg = lg.Segments(rows, max_segments=bound)
        self.ws = torch.full((max(lg.workspace_bytes(rows, slots, 1, 0), 16),), 0x7f, dtype=torch.uint8, device="cuda")
        self.dids = torch.from_numpy(self.ids).cuda()
        self.upload()

    def upload(self):
        self.table = torch.from_numpy(self.host.view(np.uint8).reshape(-1).copy()).cuda()

    def launch(self, stream=None):
        lg.build_segments(self.dids, self.slots, self.seg, self.ws, stream=stream)
        if not self.is_gated:
            lg.grouped_layer_q4g(self.dev, self.rows, self.table, self.slots, self.seg, self.group, stream=stream)
        elif self.group:
            lg.grouped_gated_layer_q4g(self.dev["gate"], self.rows, self.table, self.slots, self.seg, self.group,
                                       stream=stream, activation=self.act)
        else:
            lg.grouped_gated_layer(self.dev["gate"], self.rows, self.table, self.slots, self.seg, stream=stream,
                                   activation=self.act)

    def run(self):
        for io in self.dev.values():
            io.y.fill_(7.0)
        self.launch()
        torch.cuda.synchronize()
        return {m: io.y.clone() for m, io in self.dev.items()}

    def status(self):
        return int(self.seg.status.item())

    def reference(self, m, s, at):
        x = self.cpu[m]["x"][at // self.fan]
        sums = q4_sums if self.group else grouped_bf16
        if not self.is_gated:
            return sums(x, *self.cpu[m]["W"][m, s])
        return gated(self.act, *sums(x, *self.cpu[m]["W"]["gate", s]), *sums(x, *self.cpu[m]["W"]["up", s]))

    def check(self, got=None, skip=()):
        got = self.run() if got is None else got
        for m, (di, do, _) in self.shapes.items():
            done = np.zeros(self.rows, bool)
            for s in range(self.slots):
                at = np.nonzero(self.ids == s)[0]
                if len(at) == 0 or s in self.none or s in skip:
                    continue
                done[at] = True
                ref, slack = self.reference(m, s, at)
                close(got[m][torch.from_numpy(at).cuda()][:, :do], ref, slack, f"{m} slot {s}")
            rest = torch.from_numpy(np.nonzero(~done)[0]).cuda()
            assert bool((got[m][rest] == 7).all()), f"{m}: rows without a weight were written"
            assert bool((got[m][:, do:] == 7).all()), f"{m}: columns past d_out were written"


def one(d_in, d_out):
    return {"gate": (d_in, d_out, "m")}


def ragged(lengths, seed=0, shuffle=True):
    ids = np.repeat(np.arange(len(lengths)), lengths)
    return np.random.RandomState(seed).permutation(ids) if shuffle else ids


@forms
@pytest.mark.parametrize("rows,slots", [(1, 1), (2, 9), (16, 4), (17, 1), (40, 3), (65, 2), (130, 1), (260, 3), (700, 2),
                                        (300, 150)])
def test_rows(form, rows, slots):
    Run(form, ids_of("mixed", rows, slots, rows), slots, one(264, 136), seed=rows).check()


@forms
@pytest.mark.parametrize("lengths", [(0, 1, 0, 16, 17), (1,) * 70, (128, 0, 129, 1), (255, 257, 3, 64), (0, 0, 0, 5),
                                     (1000, 1, 1, 1), (16, 32, 64, 128)])
@pytest.mark.parametrize("shuffle", [False, True])
def test_ragged(form, lengths, shuffle):
    Run(form, ragged(lengths, 1, shuffle), len(lengths), one(136, 200), seed=len(lengths), act="gelu_tanh").check()


@forms
@pytest.mark.parametrize("d_in,d_out", [(8, 8), (24, 16), (64, 128), (72, 136), (120, 24), (264, 40), (520, 264), (1032, 72),
                                        (4104, 16)])
@pytest.mark.parametrize("rows", [3, 50, 120, 400])
def test_widths(form, d_in, d_out, rows):
    Run(form, ids_of("mixed", rows, 2, d_in), 2, one(d_in, d_out), seed=d_in + d_out).check()


@pytest.mark.parametrize("is_gated", [False, True])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("groups", [1, 2, 3, 5, 8, 9, 17, 33])
@pytest.mark.parametrize("rows", [1, 20, 100, 300])
def test_groups(is_gated, group, groups, rows):
    # every length of a group, widths that end inside a stage of every tile
    Run((is_gated, group), ids_of("mixed", rows, 2, groups), 2, one(group * groups, 72), seed=groups).check()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("kind,number,tile,lengths,d_in,d_out", [c for c in TILES if c[0].startswith("grouped")])
def test_every_tile(kind, number, tile, lengths, d_in, d_out, group):
    if not kind.endswith("q4g"):
        group = 0
    Run(("gated" in kind, group), ragged(lengths, 2), len(lengths), one(d_in, d_out), seed=tile[0], act="gelu_tanh").check()


@pytest.mark.parametrize("is_gated,group", [(True, 0), (False, 32), (True, 128)])
@pytest.mark.parametrize("rows", [3, 40, 300])
def test_a_weight_of_almost_4_gib(is_gated, group, rows):
    # offsets past 2^31 and up to the last rows of W; outputs sampled
    d_in = 8192
    d_out = (0xFFFFFF00 // (d_in // 2 if group else 2 * d_in)) // 8 * 8
    x = bf16(gen(1), rows, d_in)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    t = np.zeros((1, 7), lg.WEIGHT_Q4G_ENTRY_DTYPE)
    keep, cols = {}, ("gate", "up") if is_gated else ("gate",)
    at = torch.unique(torch.cat([torch.arange(8), torch.randint(0, d_out, (40,), generator=gen(2)),
                                 torch.arange(d_out - 24, d_out), torch.tensor([d_out // 2 - 1, d_out // 2])]))
    for c in cols:
        k = MODS.index(c)
        if group:
            W = torch.randint(0, 256, (d_out, d_in // 2), generator=g, device="cuda", dtype=torch.uint8)
            S = torch.rand(d_out, d_in // group, generator=g, device="cuda") * 0.3 * d_in ** -0.5
            t["Ws"][0, k], t["lds"][0, k] = S.data_ptr(), S.stride(0)
            w = W[at.cuda()].cpu().to(torch.int32)
            q = torch.stack([w & 15, w >> 4], -1).view(len(at), -1)
            q = torch.where(q > 7, q - 16, q)
            s = S[at.cuda()].cpu()
            keep[c] = (W, S, (q.double() * s.double().repeat_interleave(group, 1), s, group))
        else:
            W = torch.empty(d_out, d_in, dtype=torch.bfloat16, device="cuda").normal_(0, d_in ** -0.5, generator=g)
            keep[c] = (W, None, (W[at.cuda()].cpu(),))
        t["W"][0, k], t["ldw"][0, k] = W.data_ptr(), W.stride(0)
    table = torch.from_numpy(t.view(np.uint8).reshape(-1).copy()).cuda()
    y = torch.zeros(rows, d_out, dtype=torch.bfloat16, device="cuda")
    seg, ws = lg.Segments(rows, max_segments=1), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    lg.build_segments(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1, seg, ws)
    io = lg.GroupedIO(x.cuda(), y)
    if not is_gated:
        lg.grouped_layer_q4g({"gate": io}, rows, table, 1, seg, group)
    elif group:
        lg.grouped_gated_layer_q4g(io, rows, table, 1, seg, group)
    else:
        lg.grouped_gated_layer(io, rows, table, 1, seg)
    torch.cuda.synchronize()
    assert int(seg.status.item()) == 0
    sums = [(q4_sums if group else grouped_bf16)(x, *keep[c][2]) for c in cols]
    ref, slack = gated("silu", *sums[0], *sums[1]) if is_gated else sums[0]
    close(y[:, at.cuda()], ref, slack, "sampled outputs")


@forms
@pytest.mark.parametrize("fan,rows", [(2, 64), (3, 100), (8, 33), (5, 1), (2, 600)])
def test_rows_that_share_x(form, fan, rows):
    Run(form, ids_of("mixed", rows, 6, fan), 6, one(264, 200), fan=fan, seed=fan).check()


@pytest.mark.parametrize("group", GROUPS)
def test_all_projections(group):
    shapes = {"q": (256, 136, "a"), "k": (256, 40, "a"), "v": (256, 40, "a"), "o": (384, 256, "o"), "gate": (256, 520, "m"),
              "up": (256, 520, "m"), "down": (640, 256, "d")}
    for rows in (5, 90, 300):
        Run((False, group), ids_of("mixed", rows, 4, rows), 4, shapes, seed=rows, pad=8).check()


@forms
@pytest.mark.parametrize("pad", [8, 24])
def test_strides(form, pad):
    for rows in (9, 200):
        Run(form, ids_of("mixed", rows, 3, pad), 3, one(264, 136), pad=pad, seed=pad).check()


@forms
def test_slots_without_a_weight(form):
    r = Run(form, ids_of("mixed", 100, 6, 3), 6, one(264, 136), none=(1, 4))
    r.check()
    bad = int((r.ids >= 6).sum())
    assert r.status() == bad


@forms
def test_bad_entries_are_counted_and_skipped(form):
    ids = np.repeat(np.arange(8), [3, 20, 5, 1, 40, 7, 9, 2]).astype(np.int32)
    r = Run(form, ids, 8, one(264, 136))
    col = MODS.index("up" if r.is_gated else "gate")
    t, bad = r.host, [0, 1, 2]
    t["W"][0, col] += 8
    t["ldw"][1, col] -= 8
    t["ldw"][2, col] = 1 << 40
    if r.group:
        t["Ws"][3, col] = 0
        t["lds"][4, col] = r.shapes["gate"][0] // r.group - 1
        t["Ws"][5, col] += 2
        bad += [3, 4, 5]
    if r.is_gated:
        t["W"][6, col] = 0  # gate without up
        bad.append(6)
    r.upload()
    r.check(skip=bad)
    assert r.status() == len(bad)


@forms
def test_a_row_with_nan_or_infinity_reaches_no_other(form):
    ids = np.repeat(np.arange(3), [40, 1, 23]).astype(np.int32)
    r = Run(form, ids, 3, one(264, 136))
    clean = r.run()["gate"].clone()
    x = r.dev["gate"].x
    x[5, 7], x[11, :], x[39, 0], x[40, 3] = float("nan"), float("inf"), float("-inf"), float("nan")
    got = r.run()["gate"]
    hit = [5, 11, 39, 40]
    keep = torch.tensor([i for i in range(64) if i not in hit], device="cuda")
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[5, :136]).all()) and bool(torch.isnan(got[40, :136]).all())


@forms
def test_bits_repeat(form):
    r = Run(form, ids_of("mixed", 333, 5, 1), 5, one(1032, 264))
    a, b = r.run()["gate"], r.run()["gate"]
    assert torch.equal(a, b)


@forms
@pytest.mark.parametrize("rows", [12, 300])
def test_captured_and_replayed(form, rows):
    r = Run(form, ids_of("mixed", rows, 4, rows), 4, one(520, 136))
    want = r.run()["gate"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.launch()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.launch()
    y = r.dev["gate"].y
    for k in range(3):
        y.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {k}"
    r.ids[:] = r.ids[::-1].copy()  # other ids, read at the replay
    r.dids.copy_(torch.from_numpy(r.ids))
    y.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    r.check({"gate": y})


@forms
def test_on_another_stream(form):
    r = Run(form, ids_of("mixed", 90, 4, 2), 4, one(520, 136))
    want = r.run()["gate"].clone()
    r.dev["gate"].y.fill_(7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.launch(stream=side)
    side.synchronize()
    assert torch.equal(r.dev["gate"].y, want)


@forms
def test_two_calls_at_once(form):
    runs = [Run(form, ids_of("mixed", 130, 4, k), 4, one(1032, 264), seed=k) for k in range(2)]
    want = [r.run()["gate"].clone() for r in runs]
    sides = [torch.cuda.Stream() for _ in runs]
    for r, s in zip(runs, sides):
        r.dev["gate"].y.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(4):
        for r, s in zip(runs, sides):
            r.launch(stream=s)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert torch.equal(r.dev["gate"].y, w)


@forms
def test_a_segment_that_does_not_fit_the_batch(form):
    # segments built for more rows than the call: what ends past them is left alone and counted
    ids = np.repeat(np.arange(3), [30, 20, 50]).astype(np.int32)
    r = Run(form, ids, 3, one(264, 136))
    y = r.dev["gate"].y.fill_(7.0)
    lg.build_segments(r.dids, 3, r.seg, r.ws)
    r.rows = 70
    full = r.ids
    if not r.is_gated:
        lg.grouped_layer_q4g(r.dev, 70, r.table, 3, r.seg, r.group)
    elif r.group:
        lg.grouped_gated_layer_q4g(r.dev["gate"], 70, r.table, 3, r.seg, r.group)
    else:
        lg.grouped_gated_layer(r.dev["gate"], 70, r.table, 3, r.seg)
    torch.cuda.synchronize()
    assert bool((y[50:] == 7).all()) and r.status() == 1
    r.rows, r.ids = 100, np.where(full == 2, -1, full).astype(np.int32)
    r.check({"gate": y})


@forms
@pytest.mark.parametrize("bound", [2, 4])
def test_a_bound_on_the_segments(form, bound):
    ids = ids_of("mixed", 200, 4, 9)
    r = Run(form, ids, 4, one(264, 136), bound=bound)
    kept = np.unique(ids[(ids >= 0) & (ids < 4)])[:bound]
    r.check(skip=[s for s in range(4) if s not in kept])


def test_no_rows():
    for form in FORMS:
        r = Run(form, np.zeros(0, np.int32), 2, one(264, 136))
        y = r.run()["gate"]
        assert bool((y == 7).all())


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("act", ACTS)
def test_activation_over_its_range(group, act):
    # z from 0 to past both ends of sigma in fp32
    for std in (2.0 ** -60, 0.1, 30.0, 3000.0):
        Run((True, group), ids_of("mixed", 60, 2, 5), 2, one(264, 136), act=act, x_std=std, seed=int(std)).check()


def test_activation_at_infinity():
    d = 64
    x = torch.zeros(4, d, dtype=torch.bfloat16)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 3e38, -3e38, 1e30, -1e30
    W = torch.zeros(8, d, dtype=torch.bfloat16)
    W[:, 0] = 4.0  # gate: 1.2e39 is infinite in fp32
    Wu = torch.zeros(8, d, dtype=torch.bfloat16)
    Wu[:, 0] = 2.0 ** -120
    t = np.zeros((1, 7), lg.WEIGHT_ENTRY_DTYPE)
    dw, du = W.cuda(), Wu.cuda()
    for c, w in (("gate", dw), ("up", du)):
        t["W"][0, MODS.index(c)], t["ldw"][0, MODS.index(c)] = w.data_ptr(), d
    table = torch.from_numpy(t.view(np.uint8).reshape(-1).copy()).cuda()
    seg, ws = lg.Segments(4), torch.empty(64, dtype=torch.uint8, device="cuda")
    lg.build_segments(torch.zeros(4, dtype=torch.int32, device="cuda"), 1, seg, ws)
    for act in ACTS:
        h = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
        lg.grouped_gated_layer(lg.GroupedIO(x.cuda(), h), 4, table, 1, seg, activation=act)
        h = h.float().cpu()
        assert bool(torch.isinf(h[0]).all()) and bool((h[0] > 0).all())  # act(inf) = inf
        assert bool(torch.isnan(h[1]).all())                             # -inf * 0
        assert bool(((h[2] - 4e30 * 1e30 * 2.0 ** -120).abs() <= 2.0 ** -7 * h[2].abs()).all())
        assert bool((h[3] == 0).all())


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("rows", [2, 20, 300])
def test_large_rows_of_4_bit_products(group, rows):
    # magnitudes up to 2^119: no sum of a group passes the end of fp32 on its way to a finite result
    r = Run((False, group), np.zeros(rows, np.int32), 1, one(640, 72), seed=group)
    x = r.cpu["gate"]["x"]
    x.copy_((x.float().clamp(-4, 4) / 4 * 2.0 ** 119).to(torch.bfloat16))
    r.dev["gate"].x.copy_(x)
    got = r.run()
    assert bool(torch.isfinite(got["gate"][:, :72]).all())
    r.check(got)


def test_experts_gate_up_and_down_together():
    """A token's two experts: gated half and way back, 4-bit and bf16, in one captured step."""
    tokens, slots, d, f, group = 24, 5, 264, 520, 64
    d, f = 256, 576
    r = np.random.RandomState(0)
    ids = np.concatenate([r.permutation(slots)[:2] for _ in range(tokens)]).astype(np.int32)
    a = Run((True, group), ids, slots, one(d, f), fan=2, seed=3)
    b = Run((False, group), ids, slots, {"down": (f, d, "h")}, seed=4)
    b.dev["down"].x = a.dev["gate"].y

    def step():
        a.launch()
        lg.grouped_layer_q4g(b.dev, b.rows, b.table, slots, a.seg, group)

    step()
    torch.cuda.synchronize()
    a.check({"gate": a.dev["gate"].y.clone()})
    b.cpu["down"]["x"] = a.dev["gate"].y.cpu()
    want = b.dev["down"].y.clone()
    b.check({"down": want})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        b.dev["down"].y.fill_(7.0)
        a.dev["gate"].y.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.dev["down"].y, want)
