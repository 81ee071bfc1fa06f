"""Refusals of the 4-bit products with stated groups and the gated calls: every
call here fails validation, which runs before the first HIP call, so no device
is touched (the pointers are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import adapter_gemv_amd as lg
from tests.ffn_cases import TILE_SLOTS, TILES, tile_of
from tests.test_dense_abi import ALIGN, BIG, MODULE, NULL, OK, P, RANK, SHAPE, WS, _on_gpu, seg

LIN = dict(x=P, ldx=256, Wq=P, ldwq=128, Ws=P, lds=4, y=P, ldy=128, d_in=256, d_out=128, group=64, reserved=0)
GATED = dict(x=P, ldx=256, Wg=P, ldwg=256, Wu=P, ldwu=256, h=P, ldh=128, d_in=256, d_ff=128)
GATEDQ = dict(x=P, ldx=256, Wgq=P, ldwg=128, Wgs=P, ldsg=4, Wuq=P, ldwu=128, Wus=P, ldsu=4, h=P, ldh=128, d_in=256,
              d_ff=128, group=64, reserved=0)
GRP = dict(x=P, ldx=256, y=P, ldy=128, d_in=256, d_out=128, rows_per_x=1, reserved=0)
CALL = dict(mask=1, act=0, n=40, ids=P, table=P, slots=4, seg=seg(), rank=16, ws=P, ws_bytes=BIG, group=64)

# what every call with adapters refuses alike
ADAPTED = [
    (dict(x=None), {}, NULL), ({}, dict(table=None), NULL), ({}, dict(ids=None), NULL), ({}, dict(ws=None), NULL),
    ({}, dict(seg=seg(perm=None)), NULL), (dict(d_in=0), {}, SHAPE), (dict(d_in=-256), {}, SHAPE), (dict(ldx=248), {}, SHAPE),
    (dict(ldx=1 << 40), {}, SHAPE), (dict(ldx=1 << 61), {}, SHAPE), ({}, dict(n=-1), SHAPE), ({}, dict(slots=0), SHAPE),
    ({}, dict(seg=seg(max_segments=-1)), SHAPE), (dict(ldx=260), {}, ALIGN), (dict(x=P + 8), {}, ALIGN),
    ({}, dict(ws=P + 8), ALIGN), ({}, dict(rank=0), RANK), ({}, dict(rank=65), RANK), ({}, dict(ws_bytes=1000), WS),
]
Q4 = [(dict(group=g), {}, SHAPE) for g in (0, 16, 48, 96, 256, -64)]


@pytest.mark.parametrize("io,call,code", ADAPTED + Q4 + [
    (dict(Wq=None), {}, NULL), (dict(Ws=None), {}, NULL), (dict(y=None), {}, NULL), (dict(d_out=0), {}, SHAPE),
    (dict(d_out=-8), {}, SHAPE), (dict(ldy=120), {}, SHAPE), (dict(ldwq=112), {}, SHAPE), (dict(lds=3), {}, SHAPE),
    (dict(lds=1 << 40), {}, SHAPE), (dict(ldwq=1 << 60), {}, SHAPE), (dict(ldy=1 << 61), {}, SHAPE),
    (dict(d_out=1 << 25, ldy=1 << 25), dict(n=1), SHAPE), (dict(lds=1 << 26), {}, SHAPE), (dict(ldwq=1 << 26), {}, SHAPE),
    (dict(d_in=224), {}, ALIGN), (dict(d_out=124), {}, ALIGN), (dict(ldy=132), {}, ALIGN), (dict(ldwq=136), {}, ALIGN),
    (dict(y=P + 2), {}, ALIGN), (dict(Wq=P + 8), {}, ALIGN), (dict(Ws=P + 2), {}, ALIGN),
    ({}, dict(mask=0), MODULE), ({}, dict(mask=0x80), MODULE),
])
def test_linear_q4g_rejects(io, call, code):
    c = {**CALL, **call}
    arr = (lg._LinQ4GIO * 7)()
    arr[0] = lg._LinQ4GIO(*[{**LIN, **io}[k] for k, _ in lg._LinQ4GIO._fields_])
    assert lg.lib().lora_linear_layer_q4g(arr, c["mask"], c["n"], c["ids"], c["table"], c["slots"], c["seg"], c["rank"],
                                          c["ws"], c["ws_bytes"], None) == code


def test_linear_q4g_rejects_two_groups():
    arr = (lg._LinQ4GIO * 7)()
    for i, g in enumerate((64, 128)):
        arr[i] = lg._LinQ4GIO(*[{**LIN, "group": g}[k] for k, _ in lg._LinQ4GIO._fields_])
    assert lg.lib().lora_linear_layer_q4g(arr, 3, 40, P, P, 4, seg(), 16, P, BIG, None) == SHAPE


def _gated(cls, base, fn, io, call):
    c = {**CALL, **call}
    arg = cls(*[{**base, **io}[k] for k, _ in cls._fields_])
    return getattr(lg.lib(), fn)(arg, c["act"], c["n"], c["ids"], c["table"], c["slots"], c["seg"], c["rank"], c["ws"],
                                 c["ws_bytes"], None)


GATED_ALIKE = [
    (dict(h=None), {}, NULL), (dict(d_ff=0), {}, SHAPE), (dict(d_ff=-8), {}, SHAPE), (dict(ldh=120), {}, SHAPE),
    (dict(ldh=1 << 61), {}, SHAPE), (dict(d_ff=1 << 25, ldh=1 << 25), dict(n=1), SHAPE), ({}, dict(act=2), SHAPE),
    ({}, dict(act=-1), SHAPE), (dict(d_ff=124), {}, ALIGN), (dict(ldh=132), {}, ALIGN), (dict(h=P + 8), {}, ALIGN),
]


@pytest.mark.parametrize("io,call,code", ADAPTED + GATED_ALIKE + [
    (dict(Wg=None), {}, NULL), (dict(Wu=None), {}, NULL), (dict(ldwg=248), {}, SHAPE), (dict(ldwu=248), {}, SHAPE),
    (dict(ldwg=1 << 25), {}, SHAPE), (dict(ldwu=1 << 61), {}, SHAPE), (dict(d_in=252), {}, ALIGN),
    (dict(ldwg=260), {}, ALIGN), (dict(ldwu=260), {}, ALIGN), (dict(Wg=P + 8), {}, ALIGN), (dict(Wu=P + 2), {}, ALIGN),
])
def test_gated_rejects(io, call, code):
    assert _gated(lg._GatedIO, GATED, "lora_gated_layer", io, call) == code


@pytest.mark.parametrize("io,call,code", ADAPTED + GATED_ALIKE + Q4 + [
    (dict(Wgq=None), {}, NULL), (dict(Wuq=None), {}, NULL), (dict(Wgs=None), {}, NULL), (dict(Wus=None), {}, NULL),
    (dict(ldwg=112), {}, SHAPE), (dict(ldwu=112), {}, SHAPE), (dict(ldsg=3), {}, SHAPE), (dict(ldsu=3), {}, SHAPE),
    (dict(ldwg=1 << 26), {}, SHAPE), (dict(ldsu=1 << 26), {}, SHAPE), (dict(d_in=224), {}, ALIGN),
    (dict(ldwg=136), {}, ALIGN), (dict(ldwu=136), {}, ALIGN), (dict(Wgq=P + 8), {}, ALIGN), (dict(Wus=P + 2), {}, ALIGN),
])
def test_gated_q4g_rejects(io, call, code):
    assert _gated(lg._GatedQ4GIO, GATEDQ, "lora_gated_layer_q4g", io, call) == code


@pytest.mark.parametrize("fn", ["lora_grouped_layer_q4g", "lora_grouped_gated_layer", "lora_grouped_gated_layer_q4g"])
@pytest.mark.parametrize("io,call,code", [
    (dict(x=None), {}, NULL), (dict(y=None), {}, NULL), ({}, dict(table=None), NULL), ({}, dict(seg=seg(seg_offsets=None)), NULL),
    (dict(d_in=0), {}, SHAPE), (dict(d_out=0), {}, SHAPE), (dict(ldx=248), {}, SHAPE), (dict(ldy=120), {}, SHAPE),
    (dict(rows_per_x=0), {}, SHAPE), (dict(ldx=1 << 40), {}, SHAPE), (dict(ldy=1 << 61), {}, SHAPE),
    (dict(d_in=1 << 30, ldx=1 << 30), dict(n=1), SHAPE), ({}, dict(n=-1), SHAPE), ({}, dict(slots=0), SHAPE),
    ({}, dict(seg=seg(max_segments=-1)), SHAPE), (dict(d_in=252), {}, ALIGN), (dict(d_out=124), {}, ALIGN),
    (dict(ldx=260), {}, ALIGN), (dict(x=P + 8), {}, ALIGN), (dict(y=P + 8), {}, ALIGN),
    ({}, dict(mask=0), MODULE), ({}, dict(mask=0x80), MODULE), ({}, dict(act=2), SHAPE), ({}, dict(act=-1), SHAPE),
    ({}, dict(group=0), SHAPE), ({}, dict(group=48), SHAPE), ({}, dict(group=256), SHAPE), (dict(d_in=224), {}, ALIGN),
])
def test_grouped_rejects(fn, io, call, code):
    c = {**CALL, **call}
    gated, q4 = "gated" in fn, fn.endswith("q4g")
    if ("mask" in call and gated) or ("act" in call and not gated) or ("group" in call and not q4) or \
            (io.get("d_in") == 224 and not q4):
        return  # not an argument of this call
    arr = (lg._GroupedIO * 7)()
    arr[0] = lg._GroupedIO(*[{**GRP, **io}[k] for k, _ in lg._GroupedIO._fields_])
    args = [arr, c["act"] if gated else c["mask"], c["n"], c["table"], c["slots"]] + ([c["group"]] if q4 else [])
    assert getattr(lg.lib(), fn)(*args, c["seg"], None) == code


def test_no_rows_needs_no_workspace():
    arr = (lg._LinQ4GIO * 7)()
    arr[0] = lg._LinQ4GIO(*[LIN[k] for k, _ in lg._LinQ4GIO._fields_])
    assert lg.lib().lora_linear_layer_q4g(arr, 1, 0, None, P, 4, seg(), 16, None, 0, None) == OK
    no_rows = dict(n=0, ids=None, ws=None, ws_bytes=0)
    assert _gated(lg._GatedIO, GATED, "lora_gated_layer", {}, no_rows) == OK
    assert _gated(lg._GatedQ4GIO, GATEDQ, "lora_gated_layer_q4g", {}, no_rows) == OK


def test_workspace_queries():
    L = lg.lib()
    for rows, slots, rank, d in ((1, 1, 8, 256), (128, 128, 64, 8192), (5000, 7, 16, 1032)):
        one = L.lora_linear_q4g_workspace_bytes(rows, slots, rank, 2 * d, 2)
        assert one == L.lora_gated_workspace_bytes(rows, slots, rank, d)
        assert one >= L.lora_linear_workspace_bytes(rows, slots, rank, 2 * d, 2) + 4 * rows
        assert one >= L.lora_workspace_bytes(rows, slots, rank, 2 * d)
    for bad in ((-1, 4, 16, 8, 1), (4, 0, 16, 8, 1), (4, 4, 0, 8, 1), (4, 4, 65, 8, 1), (4, 4, 16, -1, 1), (4, 4, 16, 8, 0),
                (4, 4, 16, 8, 8)):
        assert L.lora_linear_q4g_workspace_bytes(*bad) == 0
    for bad in ((-1, 4, 16, 8), (4, 0, 16, 8), (4, 4, 0, 8), (4, 4, 65, 8), (4, 4, 16, -1)):
        assert L.lora_gated_workspace_bytes(*bad) == 0


def test_pack_weights_q4g():
    W = np.arange(14, dtype=np.uint64).reshape(2, 7) * 16
    t = lg.pack_weights_q4g(W, 128, W + 1000, 4)
    assert t.shape == (2, 7) and t.itemsize == 32
    assert (t["W"] == W).all() and (t["Ws"] == W + 1000).all() and (t["ldw"] == 128).all() and (t["lds"] == 4).all()


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(lg._LinQ4GIO) == 80 and ctypes.sizeof(lg._GatedIO) == 72 and ctypes.sizeof(lg._GatedQ4GIO) == 112


def _seg():
    return type("Seg", (), {"perm": _on_gpu(4, dtype="int32"), "c": lambda self: seg()})()


def _gated_args(**kw):
    d = dict(x=_on_gpu(4, 64), Wg=_on_gpu(16, 64), Wu=_on_gpu(16, 64), h=_on_gpu(4, 16), d_in=None, d_ff=None)
    d.update(kw)
    return lg.GatedIO(**d)


def _q4_args(**kw):
    d = dict(x=_on_gpu(4, 64), Wgq=_on_gpu(16, 32, dtype="uint8"), Wgs=_on_gpu(16, 2, dtype="float32"),
             Wuq=_on_gpu(16, 32, dtype="uint8"), Wus=_on_gpu(16, 2, dtype="float32"), h=_on_gpu(4, 16), group=32)
    d.update(kw)
    return lg.GatedQ4GIO(**d)


def _call_gated(io, table=7 * 32, rows=4, **kw):
    lg.gated_layer(io, rows, _on_gpu(4, dtype="int32"), _on_gpu(table, dtype="uint8"), 1, _seg(), 8, _on_gpu(16, dtype="uint8"),
                   **kw)


@pytest.mark.parametrize("io,kw,what", [
    (_gated_args, dict(x=(3, 64)), "x: fewer than 4 rows"), (_gated_args, dict(h=(4, 8)), "h: fewer than 16 columns"),
    (_gated_args, dict(Wu=(8, 64)), "Wu: fewer than 16 rows"), (_gated_args, dict(Wg=(16, 32)), "Wg: fewer than 64 columns"),
    (_q4_args, dict(Wus=(16, 1)), "Wus: fewer than 2 columns"), (_q4_args, dict(Wgq=(16, 16)), "Wgq: fewer than 32 columns"),
    (_q4_args, dict(group=16), "group must be one of"), (_q4_args, dict(group=128), "d_in must be a multiple"),
])
def test_gated_layer_refuses_short_matrices(io, kw, what):
    types = dict(Wgq="uint8", Wuq="uint8", Wgs="float32", Wus="float32")
    kw = {k: _on_gpu(*v, dtype=types.get(k, "bfloat16")) if isinstance(v, tuple) else v for k, v in kw.items()}
    with pytest.raises(ValueError, match=what):
        _call_gated(io(**kw))


def test_gated_layer_refuses_short_tables_and_unknown_activations():
    with pytest.raises(ValueError, match="table: not the 1 x 7"):
        _call_gated(_gated_args(), table=7 * 32 - 1)
    for bad in ("relu", "SILU", None, 0):
        with pytest.raises(ValueError, match="activation must be one of"):
            _call_gated(_gated_args(), activation=bad)
    with pytest.raises(ValueError, match="fewer ids"):
        _call_gated(_gated_args(x=_on_gpu(5, 64), h=_on_gpu(5, 16)), rows=5)
    with pytest.raises(TypeError):
        _call_gated(_gated_args(x=_on_gpu(4, 64, dtype="float32")))


@pytest.mark.parametrize("x,w,s,y,d_in,d_out,group,what", [
    ((4, 64), (16, 32), (16, 2), (4, 16), 96, 16, 32, "q.x: fewer than 96 columns"),
    ((4, 96), (16, 32), (16, 3), (4, 16), 96, 16, 32, "q.Wq: fewer than 48 columns"),
    ((4, 64), (16, 32), (16, 1), (4, 16), 64, 16, 32, "q.Ws: fewer than 2 columns"),
    ((4, 64), (16, 32), (8, 2), (4, 16), 64, 16, 32, "q.Ws: fewer than 16 rows"),
    ((4, 64), (16, 32), (16, 2), (4, 16), 64, 24, 32, "q.y: fewer than 24 columns"),
    ((4, 64), (16, 32), (16, 2), (4, 16), 64, 16, 48, "group must be one of"),
    ((4, 96), (16, 48), (16, 2), (4, 16), 96, 16, 64, "d_in must be a multiple"),
])
def test_linear_layer_q4g_refuses(x, w, s, y, d_in, d_out, group, what):
    io = lg.LinearQ4GIO(_on_gpu(*x), _on_gpu(*w, dtype="uint8"), _on_gpu(*s, dtype="float32"), _on_gpu(*y), group, d_in=d_in,
                        d_out=d_out)
    with pytest.raises(ValueError, match=what):
        lg.linear_layer({"q": io}, 4, _on_gpu(4, dtype="int32"), _on_gpu(7 * 32, dtype="uint8"), 1, _seg(), 8,
                        _on_gpu(16, dtype="uint8"))


def _q4g(group=32):
    return lg.LinearQ4GIO(_on_gpu(4, 128), _on_gpu(16, 64, dtype="uint8"), _on_gpu(16, 4, dtype="float32"), _on_gpu(4, 16),
                          group)


def test_linear_layer_refuses_mixed_kinds_groups_and_parts():
    args = (4, _on_gpu(4, dtype="int32"), _on_gpu(7 * 32, dtype="uint8"), 1, _seg(), 8, _on_gpu(16, dtype="uint8"))
    with pytest.raises(ValueError, match="same group"):
        lg.linear_layer({"q": _q4g(32), "k": _q4g(64)}, *args)
    x, W = _on_gpu(4, 128), _on_gpu(16, 128)
    for other in (lg.LinearIO(x, W, x), lg.LinearQ4IO(x, _on_gpu(16, 64, dtype="uint8"), _on_gpu(16, 1, dtype="float32"), x),
                  lg.LinearI8IO(x, _on_gpu(16, 128, dtype="int8"), _on_gpu(16, dtype="float32"), x)):
        for ios in ({"q": _q4g(), "k": other}, {"q": other, "k": _q4g()}):
            with pytest.raises(TypeError, match="every projection"):
                lg.linear_layer(ios, *args)
    for part in (lg.linear_shrink, lg.linear_expand):
        with pytest.raises(TypeError, match="not for LinearQ4GIO"):
            part({"q": _q4g()}, *args)


@pytest.mark.parametrize("x,y,table,fan,what", [
    ((4, 64), (4, 16), 2 * 7 * 32, 1, "weights: not the 3 x 7"), ((3, 64), (4, 16), 3 * 7 * 32, 1, "x: fewer than 4 rows"),
    ((1, 64), (4, 16), 3 * 7 * 32, 2, "x: fewer than 2 rows"), ((4, 64), (3, 16), 3 * 7 * 32, 1, "y: fewer than 4 rows"),
    ((4, 64), (4, 16), 3 * 7 * 32, 0, "rows_per_x"),
])
def test_grouped_calls_refuse_short_tables_and_matrices(x, y, table, fan, what):
    io = lg.GroupedIO(_on_gpu(*x), _on_gpu(*y), rows_per_x=fan)
    weights = _on_gpu(table, dtype="uint8")
    for call in (lambda: lg.grouped_layer_q4g({"q": io}, 4, weights, 3, _seg(), 32),
                 lambda: lg.grouped_gated_layer(io, 4, weights, 3, _seg()),
                 lambda: lg.grouped_gated_layer_q4g(io, 4, weights, 3, _seg(), 32)):
        with pytest.raises(ValueError, match=what):
            call()


@pytest.mark.parametrize("kind,number,tile,rows,d_in,d_out", TILES)
def test_batches_take_their_tile(kind, number, tile, rows, d_in, d_out):
    lengths = (rows,) if isinstance(rows, int) else rows
    slots = TILE_SLOTS if isinstance(rows, int) else len(rows)
    assert tile_of(kind, sum(lengths), slots, [(d_in, d_out)]) == (number,) + tile
    assert max(lengths) > tile[0] and max(lengths) % tile[0] and d_out > tile[1] and d_out % tile[1]


def test_every_tile_has_a_batch():
    tiles = {"gated": 5, "grouped_gated": 5, "linear_q4g": 9, "grouped_q4g": 9, "gated_q4g": 9, "grouped_gated_q4g": 9}
    for kind, n in tiles.items():
        assert sorted(c[1] for c in TILES if c[0] == kind) == list(range(n)), kind
