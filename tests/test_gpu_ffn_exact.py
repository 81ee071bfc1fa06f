"""GPU tests of the 4-bit and gated products that are tighter than a bound on every sum's error: on inputs whose sums are
exact in fp32 outputs equal the 64-bit result, rounded once; on inputs as in use the error is a rounding's."""
import numpy as np
import pytest

from tests.dense_cases import ids_of
from tests.ffn_cases import TILE_SLOTS, TILES
from tests.ffn_exact_cases import OnGpu, in_use, once, result, tight, whole
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


def batch(kind, rows):
    """(ids, slots) of a listed tile's rows."""
    if kind.startswith("grouped"):
        return np.random.RandomState(1).permutation(np.repeat(np.arange(len(rows)), rows)), len(rows)
    return ids_of("mixed", rows, TILE_SLOTS, rows), TILE_SLOTS


# every 4-bit value; the ones whose sums are smallest beside the shift's 24; none
@pytest.mark.parametrize("group,low,high", [(32, -8, 7), (64, -1, 1), (128, -8, 7), (128, 0, 0)])
@pytest.mark.parametrize("kind,number,tile,rows,d_in,d_out", TILES)
def test_scales_and_sums_in_fp32(kind, number, tile, rows, d_in, d_out, group, low, high):
    if not kind.endswith("q4g"):
        if group == 128:
            return  # bf16: twice is enough
        group = 0
    ids, slots = batch(kind, rows)
    equal(whole(KIND[kind], group, ids, slots, d_in, d_out, seed=number, act="gelu_tanh", low=low, high=high))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("low,high", [(-8, 7), (-1, 1)])
@pytest.mark.parametrize("kind,number,tile,rows,d_in,d_out", TILES)
def test_errors_are_a_roundings(kind, number, tile, rows, d_in, d_out, group, low, high):
    if not kind.endswith("q4g"):
        if (group, low) != (32, -8):
            return
        group = 0
    ids, slots = batch(kind, rows)
    rank = 0 if kind.startswith("grouped") else {32: 40, 64: 5, 128: 16}[group or 128]
    c = in_use(KIND[kind], group, ids, slots, d_in, d_out, rank, seed=number, act="gelu_tanh" if number % 2 else "silu",
               low=low, high=high)
    ref, on = result(c)
    got = OnGpu(c).run()
    assert tight(got[on], ref[on])
    assert bool(torch.isnan(got[~on]).all())


@pytest.mark.parametrize("fan", [2, 3])
@pytest.mark.parametrize("kind,group", [("grouped", 64), ("grouped_gated", 0), ("grouped_gated", 128)])
def test_rows_that_share_an_x(kind, group, fan):
    ids = ids_of("mixed", 131, 5, fan)
    equal(whole(kind, group, ids, 5, 1152, 200, fan=fan))
    c = in_use(kind, group, ids, 5, 1152, 200, fan=fan)
    ref, on = result(c)
    assert tight(OnGpu(c).run()[on], ref[on])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind,number,tile,rows,d_in,d_out", [c for c in TILES if c[0] in ("linear_q4g", "grouped_q4g")])
def test_weights_of_zeros(kind, number, tile, rows, d_in, d_out, group):
    # what the shift leaves is within the bound of the sums' errors; nothing where the scale is 0
    ids, slots = batch(kind, rows)
    c = in_use(KIND[kind], group, ids, slots, d_in, d_out, seed=number, low=0, high=0)
    for col in c.cols:
        for W, q, s in c.W[col]:
            s.copy_(torch.rand(s.shape, generator=torch.Generator().manual_seed(1)) + 0.5)
            s[::2] = 0
    got = OnGpu(c).run()
    _, on = result(c)
    scale = torch.stack([s.double().amax(1) for _, _, s in c.W["gate"]])  # the largest of an output
    x = c.x.double().abs().sum(1)[:, None]
    most = scale[torch.from_numpy(np.where(c.ids < slots, np.maximum(c.ids, 0), 0) if not c.adapted else np.zeros_like(c.ids))]
    left = got[on].double().abs()
    assert bool((left[:, ::2] == 0).all())
    assert bool((left <= (2 * (2 * group + 4) * 2.0 ** -24 * 48 * (1 + 2.0 ** -8)) * (x * most)[on]).all())
    print(f"[left] {kind} {number} group {group}: {float((left / (x * most + 1e-30)[on]).max()):.3g} of the scale times sum |x|")
