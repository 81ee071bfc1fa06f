"""Refusals of the 4-bit and gated calls by slot, beside those of test_ffn_abi.py: every call here fails before the
device is touched."""
import pytest

import adapter_gemv_amd as lg
from tests.test_dense_abi import _on_gpu, seg


@pytest.mark.parametrize("rows,held", [(4, 3), (4, 1), (1, 0), (4096, 10)])
def test_grouped_calls_refuse_segments_of_a_smaller_batch(rows, held):
    # buffers for `held` rows: the kernels would read offsets of up to min(rows, slots) segments
    s = type("Seg", (), {"perm": _on_gpu(held, dtype="int32"), "c": lambda self: seg()})()
    io, weights = lg.GroupedIO(_on_gpu(rows, 64), _on_gpu(rows, 16)), _on_gpu(3 * 7 * 32, dtype="uint8")
    for call in (lambda: lg.grouped_layer_q4g({"q": io}, rows, weights, 3, s, 32),
                 lambda: lg.grouped_gated_layer(io, rows, weights, 3, s),
                 lambda: lg.grouped_gated_layer_q4g(io, rows, weights, 3, s, 32)):
        with pytest.raises(ValueError, match="Segments buffers too small"):
            call()
