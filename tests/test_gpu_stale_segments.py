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
