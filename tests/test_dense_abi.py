"""Refusals of the int8 base projection and the grouped products: every call
here fails validation, which runs before the first HIP call, so no device is
touched (the pointers are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import adapter_gemv_amd as lg
from tests.dense_cases import GROUPED_TILES, LINEAR_SLOTS, LINEAR_TILES, tile_of

OK, NULL, SHAPE, RANK, ALIGN, WS, MODULE = range(7)
P = 0x10000
BIG = 1 << 40


def seg(**kw):
    d = dict(perm=P, seg_offsets=P, seg_adapter=P, num_segments=P, tile_counts=P, status=P)
    d.update(kw)
    return lg._Seg(**d)


LIN = dict(x=P, ldx=256, Wq=P, ldwq=256, Ws=P, y=P, ldy=128, d_in=256, d_out=128)
GRP = dict(x=P, ldx=256, y=P, ldy=128, d_in=256, d_out=128, rows_per_x=1, reserved=0)
CALL = dict(mask=1, n=40, ids=P, table=P, slots=4, seg=seg(), rank=16, ws=P, ws_bytes=BIG)


@pytest.mark.parametrize("fn", ["lora_linear_layer_i8", "lora_linear_shrink_i8", "lora_linear_expand_i8"])
@pytest.mark.parametrize("io,call,code", [
    (dict(x=None), {}, NULL), (dict(Wq=None), {}, NULL), (dict(Ws=None), {}, NULL), (dict(y=None), {}, NULL),
    ({}, dict(table=None), NULL), ({}, dict(ids=None), NULL), ({}, dict(ws=None), NULL),
    ({}, dict(seg=seg(perm=None)), NULL),
    (dict(d_in=0), {}, SHAPE), (dict(d_out=-8), {}, SHAPE), (dict(ldx=248), {}, SHAPE), (dict(ldy=120), {}, SHAPE),
    (dict(ldwq=240), {}, SHAPE), (dict(d_in=131080, ldx=131080, ldwq=131088), {}, SHAPE),
    (dict(d_out=1 << 25, ldy=1 << 25), {}, SHAPE), (dict(ldwq=1 << 60), {}, SHAPE), (dict(ldx=1 << 40), {}, SHAPE),
    (dict(ldx=1 << 61), {}, SHAPE), (dict(ldy=1 << 61), {}, SHAPE), (dict(d_out=(1 << 29) + 8, ldy=(1 << 29) + 8), {}, SHAPE),
    (dict(d_in=8, ldx=8, ldwq=16, d_out=1 << 25, ldy=1 << 25), dict(n=1), SHAPE),
    ({}, dict(n=-1), SHAPE), ({}, dict(slots=0), SHAPE), ({}, dict(seg=seg(max_segments=-1)), SHAPE),
    (dict(d_in=252), {}, ALIGN), (dict(d_out=124), {}, ALIGN), (dict(ldx=260), {}, ALIGN), (dict(ldy=132), {}, ALIGN),
    (dict(ldwq=264), {}, ALIGN), (dict(x=P + 8), {}, ALIGN), (dict(y=P + 2), {}, ALIGN), (dict(Wq=P + 8), {}, ALIGN),
    (dict(Ws=P + 4), {}, ALIGN), ({}, dict(ws=P + 8), ALIGN),
    ({}, dict(rank=0), RANK), ({}, dict(rank=65), RANK),
    ({}, dict(mask=0), MODULE), ({}, dict(mask=0x80), MODULE),
    ({}, dict(ws_bytes=1000), WS),
])
def test_linear_i8_rejects(fn, io, call, code):
    c = {**CALL, **call}
    arr = (lg._LinI8IO * 7)()
    arr[0] = lg._LinI8IO(*[{**LIN, **io}[k] for k, _ in lg._LinI8IO._fields_])
    got = getattr(lg.lib(), fn)(arr, c["mask"], c["n"], c["ids"], c["table"], c["slots"], c["seg"], c["rank"], c["ws"],
                                c["ws_bytes"], None)
    assert got == code


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("io,call,code", [
    (dict(x=None), {}, NULL), (dict(y=None), {}, NULL), ({}, dict(table=None), NULL),
    ({}, dict(seg=seg(seg_offsets=None)), NULL),
    (dict(d_in=0), {}, SHAPE), (dict(d_out=0), {}, SHAPE), (dict(ldx=248), {}, SHAPE), (dict(ldy=120), {}, SHAPE),
    (dict(rows_per_x=0), {}, SHAPE), (dict(rows_per_x=-2), {}, SHAPE), (dict(ldx=1 << 40), {}, SHAPE),
    (dict(ldy=1 << 40), {}, SHAPE), (dict(ldx=1 << 61), {}, SHAPE), (dict(ldy=1 << 61), {}, SHAPE),
    (dict(d_in=1 << 30, ldx=1 << 30), dict(n=1), SHAPE), (dict(d_out=1 << 30, ldy=1 << 30), dict(n=1), SHAPE),
    ({}, dict(n=-1), SHAPE), ({}, dict(slots=0), SHAPE),
    ({}, dict(seg=seg(max_segments=-1)), SHAPE),
    (dict(d_in=252), {}, ALIGN), (dict(d_out=124), {}, ALIGN), (dict(ldx=260), {}, ALIGN), (dict(ldy=132), {}, ALIGN),
    (dict(x=P + 8), {}, ALIGN), (dict(y=P + 8), {}, ALIGN),
    ({}, dict(mask=0), MODULE), ({}, dict(mask=0x80), MODULE), ({}, dict(mask=1 << 16), MODULE),
])
def test_grouped_rejects(int8, io, call, code):
    c = {**CALL, **call}
    arr = (lg._GroupedIO * 7)()
    arr[0] = lg._GroupedIO(*[{**GRP, **io}[k] for k, _ in lg._GroupedIO._fields_])
    if int8:
        got = lg.lib().lora_grouped_layer_i8(arr, c["mask"], c["n"], c["table"], c["slots"], c["seg"], c["ws"],
                                             c["ws_bytes"], None)
    else:
        got = lg.lib().lora_grouped_layer(arr, c["mask"], c["n"], c["table"], c["slots"], c["seg"], None)
    assert got == code


@pytest.mark.parametrize("io,call,code", [
    ({}, dict(ws=None), NULL), ({}, dict(ws=P + 8), ALIGN), ({}, dict(ws_bytes=100), WS),
    (dict(d_in=131080, ldx=131080), {}, SHAPE),
])
def test_grouped_i8_rejects(io, call, code):
    c = {**CALL, **call}
    arr = (lg._GroupedIO * 7)()
    arr[0] = lg._GroupedIO(*[{**GRP, **io}[k] for k, _ in lg._GroupedIO._fields_])
    assert lg.lib().lora_grouped_layer_i8(arr, c["mask"], c["n"], c["table"], c["slots"], c["seg"], c["ws"], c["ws_bytes"],
                                          None) == code


def test_workspace_queries():
    L = lg.lib()
    full = L.lora_linear_i8_workspace_bytes(128, 128, 64, 8192, 1)
    assert full > L.lora_linear_workspace_bytes(128, 128, 64, 8192, 1)
    assert full >= L.lora_workspace_bytes(128, 128, 64, 8192)
    assert L.lora_linear_i8_workspace_bytes(128, 128, 64, 16384, 2) > full
    for bad in ((-1, 4, 16, 8, 1), (4, 0, 16, 8, 1), (4, 4, 0, 8, 1), (4, 4, 65, 8, 1), (4, 4, 16, -1, 1), (4, 4, 16, 8, 0),
                (4, 4, 16, 8, 8)):
        assert L.lora_linear_i8_workspace_bytes(*bad) == 0
    assert L.lora_grouped_workspace_bytes(100, 4, 8192, 1) >= 100 * (8192 + 4)
    # room for each of n matrices' rows, scales and alignment, whatever the sum's split
    for n, rows, dims in ((7, 1, [8] * 7), (3, 17, [8, 24, 1032])):
        need = sum(-(-rows * (-(-d // 16) * 16) // 256) * 256 + -(-rows * 4 // 256) * 256 for d in dims)
        assert L.lora_grouped_workspace_bytes(rows, 4, sum(dims), n) >= need
    for bad in ((-1, 4, 8, 1), (4, 0, 8, 1), (4, 4, -1, 1), (4, 4, 8, 0), (4, 4, 8, 8)):
        assert L.lora_grouped_workspace_bytes(*bad) == 0


def test_pack_weights():
    W = np.arange(14, dtype=np.uint64).reshape(2, 7) * 16
    t = lg.pack_weights(W, 256, W + 1000)
    assert t.shape == (2, 7) and t.itemsize == 32
    assert (t["W"] == W).all() and (t["Ws"] == W + 1000).all() and (t["ldw"] == 256).all()
    assert (lg.pack_weights(W, 8)["Ws"] == 0).all()


def test_struct_sizes_match_the_header():
    # lora_linear_i8_io_t: 7 words of 8 bytes and two ints; lora_grouped_io_t: 4 words and four ints
    assert ctypes.sizeof(lg._LinI8IO) == 64 and ctypes.sizeof(lg._GroupedIO) == 48


def test_binding_checks_its_arguments():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    io = lg.GroupedIO(x, x)
    with pytest.raises(ValueError):  # not on the GPU
        lg.grouped_layer({"q": io}, 4, x, 1, None)
    with pytest.raises(TypeError):
        lg.linear_layer({"q": lg.LinearI8IO(x, x, x, x), "k": lg.LinearIO(x, x, x)}, 4, x, x, 1, None, 8, x)


def _on_gpu(*shape, dtype="bfloat16"):
    """A CPU tensor that says it is on GPU 0: for checks that end before the device is touched."""
    torch = pytest.importorskip("torch")

    class OnGpu(torch.Tensor):
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 0

    return torch.zeros(*shape, dtype=getattr(torch, dtype)).as_subclass(OnGpu)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("x,y,table,d_in,d_out,fan,what", [
    ((4, 16), (4, 16), 2 * 7 * 32, 16, 16, 1, "weights: not the 3 x 7"),    # one slot short
    ((4, 16), (4, 16), 3 * 7 * 32 - 1, 16, 16, 1, "weights: not the 3 x 7"),
    ((4, 16), (4, 16), 0, 16, 16, 1, "weights: not the 3 x 7"),
    ((4, 16), (4, 16), 3 * 7 * 32, 24, 16, 1, "q.x: fewer than 24 columns"),
    ((1, 8), (4, 16), 3 * 7 * 32, 16, 16, 4, "q.x: fewer than 16 columns"),  # a single row: its stride says nothing
    ((4, 16), (4, 16), 3 * 7 * 32, 16, 24, 1, "q.y: fewer than 24 columns"),
    ((3, 16), (4, 16), 3 * 7 * 32, 16, 16, 1, "q.x: fewer than 4 rows"),
    ((1, 16), (4, 16), 3 * 7 * 32, 16, 16, 2, "q.x: fewer than 2 rows"),
    ((4, 16), (3, 16), 3 * 7 * 32, 16, 16, 1, "q.y: fewer than 4 rows"),
])
def test_grouped_layer_refuses_short_tables_and_matrices(int8, x, y, table, d_in, d_out, fan, what):
    io = lg.GroupedIO(_on_gpu(*x), _on_gpu(*y), d_in=d_in, d_out=d_out, rows_per_x=fan)
    with pytest.raises(ValueError, match=what):
        lg.grouped_layer({"q": io}, 4, _on_gpu(table, dtype="uint8"), 3, None, int8=int8)


@pytest.mark.parametrize("x,w,y,table,d_in,d_out,what", [
    ((4, 16), (16, 16), (4, 16), 2 * 7 * 32, 16, 16, "table: not the 3 x 7"),
    ((4, 16), (16, 16), (4, 16), 3 * 7 * 32, 24, 16, "q.x: fewer than 24 columns"),
    ((4, 32), (16, 16), (4, 16), 3 * 7 * 32, 24, 16, "q.Wq: fewer than 24 columns"),
    ((4, 16), (16, 16), (4, 16), 3 * 7 * 32, 16, 24, "q.y: fewer than 24 columns"),
    ((4, 16), (16, 16), (4, 24), 3 * 7 * 32, 16, 24, "q.Wq: fewer than 24 rows"),
    ((3, 16), (16, 16), (4, 16), 3 * 7 * 32, 16, 16, "q.x: fewer than 4 rows"),
])
def test_linear_layer_i8_refuses_short_tables_and_matrices(x, w, y, table, d_in, d_out, what):
    io = lg.LinearI8IO(_on_gpu(*x), _on_gpu(*w, dtype="int8"), _on_gpu(w[0], dtype="float32"), _on_gpu(*y), d_in=d_in,
                       d_out=d_out)
    seg = type("Seg", (), {"perm": None})()
    with pytest.raises(ValueError, match=what):
        lg.linear_layer({"q": io}, 4, _on_gpu(4, dtype="int32"), _on_gpu(table, dtype="uint8"), 3, seg, 8,
                        _on_gpu(64, dtype="uint8"))


def test_tables_in_pieces_are_refused():
    wide = _on_gpu(3 * 7, 64, dtype="uint8")[:, :32]
    x = _on_gpu(4, 16)
    with pytest.raises(ValueError, match="weights: not the 3 x 7"):
        lg.grouped_layer({"q": lg.GroupedIO(x, x)}, 4, wide, 3, None)


class _LikeLinear:
    def __init__(self, **kw):
        self.__dict__.update(kw)


def _linear_call(ios):
    held = type("Seg", (), {"perm": _on_gpu(4, dtype="int32"), "c": lambda self: seg()})()
    lg.linear_layer(ios, 4, _on_gpu(4, dtype="int32"), _on_gpu(7 * 32, dtype="uint8"), 1, held, 8, _on_gpu(16, dtype="uint8"),
                    stream=_LikeLinear(cuda_stream=0))


def test_any_object_with_the_attributes_is_a_bf16_projection():
    # it gets as far as the library's own check of the workspace (host only)
    x, W = _on_gpu(4, 16), _on_gpu(16, 16)
    like = _LikeLinear(x=x, W=W, y=x, d_in=16, d_out=16)
    sub = type("Sub", (lg.LinearIO,), {})(x, W, x)
    for ios in ({"q": like}, {"q": sub}, {"q": lg.LinearIO(x, W, x), "k": like}, {"q": like, "k": lg.LinearIO(x, W, x)},
                {"q": None, "k": like}):
        with pytest.raises(lg.LoraError, match="WORKSPACE"):
            _linear_call(ios)


def test_projections_of_two_kinds_are_refused():
    x, W, q = _on_gpu(4, 128), _on_gpu(128, 128), _on_gpu(128, 64, dtype="uint8")
    s = _on_gpu(128, 1, dtype="float32")
    kinds = [_LikeLinear(x=x, W=W, y=x, d_in=128, d_out=128), lg.LinearIO(x, W, x), lg.LinearQ4IO(x, q, s, x),
             lg.LinearI8IO(x, _on_gpu(128, 128, dtype="int8"), _on_gpu(128, dtype="float32"), x)]
    for i, a in enumerate(kinds):
        for j, b in enumerate(kinds):
            if i != j and max(i, j) >= 2:
                with pytest.raises(TypeError, match="every projection"):
                    _linear_call({"q": a, "k": b})


@pytest.mark.parametrize("tile,rows,d_in,d_out", LINEAR_TILES)
def test_int8_base_batches_take_their_tile(tile, rows, d_in, d_out):
    assert tile_of("linear_i8", rows, LINEAR_SLOTS, [(d_in, d_out)]) == tile
    assert rows > tile[0] and rows % tile[0] and d_out > tile[1] and d_out % tile[1]


@pytest.mark.parametrize("kind", ["grouped", "grouped_i8"])
@pytest.mark.parametrize("tile,lengths,d_in,d_out", GROUPED_TILES)
def test_grouped_batches_take_their_tile(kind, tile, lengths, d_in, d_out):
    assert tile_of(kind, sum(lengths), len(lengths), [(d_in, d_out)]) == tile
    assert max(lengths) > tile[0] and max(lengths) % tile[0] and d_out > tile[1] and d_out % tile[1]


def test_every_tile_has_a_batch():
    tiles = [(16, 64), (32, 64), (64, 64), (128, 96), (128, 128), (256, 256)]
    for cases in (LINEAR_TILES, GROUPED_TILES):
        assert sorted({c[0] for c in cases}) == tiles
