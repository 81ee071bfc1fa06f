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
