"""GPU tests of calls whose segments are not the batch's (built from other ids, for a longer batch, or damaged): what is
written stays inside the batch and inside what the segments hold, and each segment that does not fit is counted once."""
import numpy as np
import pytest

from tests.parity import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import adapter_gemv_amd as lg  # noqa: E402
from tests import test_gpu_ffn_adapted as adapted  # noqa: E402
from tests import test_gpu_ffn_grouped as grouped  # noqa: E402
from tests import test_gpu_linear_i8 as i8  # noqa: E402


@pytest.fixture(autouse=True)
def _name_case(request):
    note(request.node.nodeid)


@pytest.mark.parametrize("rows,kept", [(90, 37), (600, 300)])
def test_int8_base_with_ids_other_than_the_segments(rows, kept):
    # rows that get a slot after the segments were built have no place in the order of the slots; whatever the workspace
    # held there before, they stay unwritten (row `kept` would have had a v that no launch wrote)
    r = i8.Run(rows, 3, {"q": (264, 136, "a")}, 16, seed=5)
    r.ids = np.sort(np.random.RandomState(3).randint(0, 3, rows)).astype(np.int32)
    r.ids[kept:] = -1
    r.dids.copy_(torch.from_numpy(r.ids))
    lg.build_segments(r.dids, 3, r.seg, r.ws)
    r.dids[kept:] = 0
    r.ws[:r.ws.numel() // 4 * 4].view(torch.int32).fill_(kept)
    r.dev["q"].y.fill_(float("nan"))
    lg.linear_layer(*r.args())
    torch.cuda.synchronize()
    assert bool(torch.isnan(r.dev["q"].y[kept:]).all())
    ref, slack = r.reference("q")
    i8.close(r.out()["q"][:kept], ref[:kept], slack[:kept], "q")


def longer(r, lengths, rows):
    """Segments of these lengths, built for all their rows, and then a call for `rows`: the ones that do not fit."""
    r.ids = np.repeat(np.arange(len(lengths)), lengths).astype(np.int32)
    r.dids.copy_(torch.from_numpy(r.ids))
    lg.build_segments(r.dids, r.slots, r.seg, r.ws)
    return [s for s, end in enumerate(np.cumsum(lengths)) if end > rows]


LENGTHS = [(40, 30, 20, 10), (3, 90, 4, 3), (64, 8, 7, 21)]


@adapted.forms
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("rows", [20, 71, 97])
def test_segments_of_a_longer_batch_are_counted_once(form, lengths, rows):
    # (71 and 97 rows: by the grouped shrink, whose long segments two kinds of work items look at)
    r = adapted.Run(form, sum(lengths), len(lengths), adapted.one(264, 136), 16)
    out = longer(r, lengths, rows)
    r.call(rows=rows)
    torch.cuda.synchronize()
    assert r.status() == len(out) > 0


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("rows", [20, 71, 97])
@pytest.mark.parametrize("call", ["int8", "delta", "expand"])
def test_older_calls_count_them_once(call, lengths, rows):
    r = i8.Run(sum(lengths), len(lengths), {"q": (264, 136, "a")}, 16)
    out = longer(r, lengths, rows)
    r.rows, io = rows, r.dev["q"]
    if call == "int8":
        lg.linear_layer(*r.args())
    elif call == "delta":
        lg.apply_layer({"q": lg.ModuleIO(io.x, io.y, d_in=264, d_out=136)}, rows, r.table, r.slots, r.seg, 16, r.ws)
    else:
        v = torch.ones(rows, 16, device="cuda")
        lg.expand(v, r.table, r.slots, 7, 0, r.seg, 16, io.y[:rows], r.ws)
    torch.cuda.synchronize()
    assert int(r.seg.status.item()) == len(out) > 0


# An end below the smallest length's start wraps a 32-bit difference round to a large length: segment 1 is (40, END),
# segment 2 (END, 90).
ENDS = [-2 ** 31, -2 ** 31 + 39, -1, 0, 40, 101, 2 ** 31 - 1]
FOUR = (40, 30, 20, 10)


def damaged(r, end):
    """(segments that do not fit, for each row the segments that hold it): an end of 0 or 40 makes segment 2 one that
    fits, over rows of others."""
    longer(r, FOUR, 100)
    r.seg.seg_offsets[2] = end
    offsets = [0, 40, end, 90, 100]
    fit = [s for s in range(4) if 0 <= offsets[s] < offsets[s + 1] <= 100]
    return [s for s in range(4) if s not in fit], [[s for s in fit if offsets[s] <= b < offsets[s + 1]] for b in range(100)]


@adapted.forms
@pytest.mark.parametrize("end", ENDS)
def test_damaged_offsets_with_adapters(form, end):
    r = adapted.Run(form, 100, 4, adapted.one(264, 136), 16, pad=8)
    bad, _ = damaged(r, end)
    r.out("gate").fill_(7.0)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == len(bad) > 0
    y = r.out("gate")[:, :136]
    assert bool(torch.isfinite(y).all()) and bool((r.out("gate")[:, 136:] == 7).all())


@grouped.forms
@pytest.mark.parametrize("end", ENDS)
def test_damaged_offsets_by_slot(form, end):
    r = grouped.Run(form, np.repeat(np.arange(4), FOUR), 4, grouped.one(264, 136), pad=8)
    bad, holds = damaged(r, end)
    r.dev["gate"].y.fill_(7.0)
    if r.is_gated and r.group:
        lg.grouped_gated_layer_q4g(r.dev["gate"], 100, r.table, 4, r.seg, r.group)
    elif r.is_gated:
        lg.grouped_gated_layer(r.dev["gate"], 100, r.table, 4, r.seg)
    else:
        lg.grouped_layer_q4g(r.dev, 100, r.table, 4, r.seg, r.group)
    torch.cuda.synchronize()
    assert r.status() == len(bad) > 0
    y = r.dev["gate"].y
    assert bool((y[:, 136:] == 7).all())
    # (segments that overlap hold more rows than the batch, and more tiles than the grid has blocks for)
    for s in range(4) if all(len(h) <= 1 for h in holds) else ():
        at = np.array([b for b in range(100) if holds[b] == [s]], int)
        if len(at):
            ref, slack = r.reference("gate", s, at)
            grouped.close(y[torch.from_numpy(at).cuda()][:, :136], ref, slack, f"segment {s}")
    none = torch.tensor([b for b in range(100) if not holds[b]], dtype=torch.long, device="cuda")
    assert bool((y[none] == 7).all())


@pytest.mark.parametrize("end", ENDS)
def test_damaged_offsets_of_the_older_calls(end):
    r = i8.Run(100, 4, {"q": (264, 136, "a")}, 16)
    bad, holds = damaged(r, end)
    io = r.dev["q"]
    io.y.fill_(7.0)
    lg.apply_layer({"q": lg.ModuleIO(io.x, io.y, d_in=264, d_out=136)}, 100, r.table, r.slots, r.seg, 16, r.ws)
    torch.cuda.synchronize()
    assert int(r.seg.status.item()) == len(bad) > 0
    same = (io.y == 7).all(1).cpu()
    assert [bool(v) for v in same] == [not h for h in holds]
    r.seg.status.zero_()
    lg.linear_layer(*r.args())
    torch.cuda.synchronize()
    assert int(r.seg.status.item()) == len(bad) and bool(torch.isfinite(io.y).all())
