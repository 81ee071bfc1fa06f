"""GPU tests of the 4-bit and gated products on inputs whose sums are exact in fp32: outputs equal the 64-bit result,
rounded once."""
import numpy as np
import pytest

from tests.dense_cases import ids_of
from tests.ffn_cases import TILE_SLOTS, TILES
from tests.ffn_exact_cases import OnGpu, once, whole
from tests.parity import note

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)


@pytest.fixture(autouse=True)
def _name_case(request):
    note(request.node.nodeid)


def equal(c):
    want, on = once(c)
    got = OnGpu(c).run()
    bad = got[on].view(torch.int16) != want[on].view(torch.int16)
    bad &= (got[on] != 0) | (want[on] != 0)  # zeros of either sign
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outputs differ; first {got[on][bad][:4]} {want[on][bad][:4]}"
    assert bool(torch.isnan(got[~on]).all())


KIND = {"linear_q4g": "linear", "gated_q4g": "gated", "gated": "gated", "grouped_q4g": "grouped",
        "grouped_gated": "grouped_gated", "grouped_gated_q4g": "grouped_gated"}


# ranks that take the product's two forms (up to 32, above)
@pytest.mark.parametrize("group,rank", [(32, 40), (64, 5), (128, 16)])
@pytest.mark.parametrize("kind,number,tile,rows,d_in,d_out", [c for c in TILES if not c[0].startswith("grouped")])
def test_every_bit_of_v(kind, number, tile, rows, d_in, d_out, group, rank):
    group = group if kind.endswith("q4g") else 0
    ids = ids_of("mixed", rows, TILE_SLOTS, rows)
    if "gated" in kind:  # without its delta a gate is not one of 90 and more
        ids %= TILE_SLOTS
    equal(whole(KIND[kind], group, ids, TILE_SLOTS, d_in, d_out, rank, seed=number))


@pytest.mark.parametrize("rows", [20, 100])
def test_a_v_that_is_infinite(rows):
    # A x past the type gives infinite outputs, not NaN, and none in other rows
    c = whole("linear", 32, np.zeros(rows, np.int32), 1, 256, 64, 1)
    want, _ = once(c)
    c.A["gate"][0][:, 5] = 3e38
    c.x[3:7, 5] = 4
    got = OnGpu(c).run()
    assert bool((got[3:7] == float("inf")).all())
    got[3:7] = want[3:7]
    assert torch.equal(got, want)
