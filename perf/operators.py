"""Measured operators: the int8 base projection with the adapter delta
(linear_i8), and the products grouped by slot with ragged row counts in bf16
(grouped) and int8 (grouped_i8).

``own`` selects the form ``run`` takes: False, elementary torch operations in
32 bits, rounded once at the end; True, the calls of ``adapter_gemv_amd``.

Formulas (row b of the batch, a = its slot id):

* linear_i8: s_b = max|x_b| / 127, q_b = rint(127 x_b / max|x_b|),
  y_b = bf16( s_b * Ws[n] * sum_k q_b[k] Wq[n][k]  +  scale_a * B_a (A_a x_b) );
  rows with a negative id get the first term only.
* grouped: y_b = bf16( W_a x_{b // fan} ), rows with a negative id untouched.
* grouped_i8: the same with W_a = Ws_a[n] * Wq_a[n][k] and x quantised per row
  as above.
"""
import math

import numpy as np
import torch

own = False

# Projections of a layer: (input, output) widths by name, and which share x.
_MODS = {"q": ("d", "d"), "k": ("d", "kv"), "v": ("d", "kv"), "o": ("d", "d"),
         "gate": ("d", "ffn"), "up": ("d", "ffn"), "down": ("ffn", "d")}
_SHARE = {"q": "attn", "k": "attn", "v": "attn", "o": "o", "gate": "mlp", "up": "mlp", "down": "down"}


def _case(name, op, mods, rows, slots, ids, d=8192, kv=1024, ffn=28672, rank=0, base=0.0, fan=1, batch=1):
    c = {"op": op, "mods": mods, "rows": rows, "slots": slots, "ids": ids, "d": d, "kv": kv, "ffn": ffn, "rank": rank,
         "base": base, "fan": fan, "batch": batch}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the smallest decode call: 16 rows, 4 adapters of rank 8 on one 256 x 256 projection (launch latency)
        _case("linear-i8-tiny", "linear_i8", "q", 16, 4, "uniform", d=256, rank=8),
        # one token of one request on a 70B attention block: the int8 weights read once
        _case("linear-i8-one-row", "linear_i8", "q,k,v,o", 1, 1, "uniform", rank=16),
        # the worst decode step: every projection, 128 rows with 128 different adapters of rank 64
        _case("linear-i8-layer-decode", "linear_i8", "q,k,v,o,gate,up,down", 128, 128, "distinct", rank=64),
        # skewed decode traffic: 256 rows over 512 resident adapters, some rows without one
        _case("linear-i8-zipf", "linear_i8", "q,k,v,o", 256, 512, "zipf", rank=32, base=0.1),
        # odd widths, odd rank and a ragged batch on every projection
        _case("linear-i8-odd", "linear_i8", "q,k,v,o,gate,up,down", 37, 19, "uniform", d=1032, kv=72, ffn=2056, rank=5,
              base=0.1),
        # prefill: 32 sequences of 128 to 2048 tokens, each with its own adapter (compute bound)
        _case("linear-i8-prefill", "linear_i8", "q,o", 0, 32, "runs", rank=16),
        # the smallest grouped call: 16 rows over 4 slots of 256 x 256 weights
        _case("grouped-tiny", "grouped", "q", 16, 4, "uniform", d=256),
        # decode rows spread over 32 merged adapters: every slot's weight read once
        _case("grouped-decode", "grouped", "q", 128, 32, "uniform"),
        # odd widths, ragged groups, three slots for every token
        _case("grouped-odd", "grouped", "q,k,v,o,gate,up,down", 333, 7, "uniform", d=1032, kv=72, ffn=2056, fan=3,
              base=0.05),
        # prefill sequences on 32 merged adapters (compute bound)
        _case("grouped-prefill", "grouped", "q", 0, 32, "runs"),
        # decode through experts: 64 tokens, two of 8 int8 experts each, the two input projections of the MLP
        _case("grouped-i8-decode", "grouped_i8", "gate,up", 128, 8, "uniform", fan=2),
        # prefill through int8 weights, two projections
        _case("grouped-i8-prefill", "grouped_i8", "q,o", 0, 32, "runs"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limit = {}
    for c in listed():
        w = work(c)
        f, b = limit.get(c["op"], (0, 0))
        limit[c["op"]] = (max(f, w["flops"]), max(b, w["bytes"]))
    while True:
        op = rng.choice(["linear_i8", "linear_i8", "grouped", "grouped_i8"])
        mods = rng.choice(["q", "k", "q,k,v,o", "gate,up", "down", "q,o", "q,k,v,o,gate,up,down"])
        d = 8 * _log(rng, 32, 1024)
        kv = 8 * _log(rng, 4, max(5, d // 8))
        ffn = 8 * _log(rng, max(8, d // 8), max(9, min(3584, d // 2)))
        ids = rng.choice(["uniform", "zipf", "runs"])
        rows = 0 if ids == "runs" else _log(rng, 1, 2048)
        slots = _log(rng, 1, 32 if ids == "runs" else 256)
        c = _case("", op, mods, rows, slots, ids, d=d, kv=kv, ffn=ffn,
                  rank=rng.choice([1, 5, 8, 12, 16, 32, 48, 64]) if op == "linear_i8" else 0,
                  base=rng.choice([0.0, 0.0, 0.1]), fan=1 if ids == "runs" or op == "linear_i8" else rng.choice([1, 1, 2, 3]),
                  batch=rng.randrange(1 << 30))
        held = sum(i * o for _, i, o in _shapes(c)) * slots * 4  # the plain form's 32-bit weights of every slot
        f, b = limit[op]
        w = work(c)
        if w["flops"] <= f and w["bytes"] <= b and (op == "linear_i8" or held <= 16e9):
            return c


def _shapes(c):
    return [(m, c[_MODS[m][0]], c[_MODS[m][1]]) for m in c["mods"].split(",")]


def _ids(c):
    """The batch's slot ids (host int32): what the scheduler formed."""
    r = np.random.RandomState(c["batch"] % (1 << 31))
    n, s = c["rows"], c["slots"]
    if c["ids"] == "runs":
        ids = np.repeat(r.permutation(s), r.randint(128, 2049, s))
    elif c["ids"] == "distinct":
        ids = r.permutation(s)[:n]
    elif c["ids"] == "zipf":
        p = 1.0 / np.arange(1, s + 1) ** 1.1
        ids = r.choice(r.permutation(s), n, p=p / p.sum())
    elif c["fan"] > 1 and c["fan"] <= s:  # a token's slots differ
        ids = np.concatenate([r.permutation(s)[:c["fan"]] for _ in range(-(-n // c["fan"]))])[:n]
    else:
        ids = r.randint(0, s, n)
    ids = ids.astype(np.int32)
    if c["base"]:
        ids[r.random_sample(ids.size) < c["base"]] = -1
    return ids


def work(c):
    ids = _ids(c)
    n, on, distinct = ids.size, int((ids >= 0).sum()), int(np.unique(ids[ids >= 0]).size)
    i8 = c["op"] != "grouped"
    b = f = 0
    seen = set()
    for m, di, do in _shapes(c):
        if _SHARE[m] not in seen:
            seen.add(_SHARE[m])
            b += 2 * di * (n if c["op"] == "linear_i8" else -(-n // c["fan"]))
        if c["op"] == "linear_i8":
            b += di * do + 4 * do + 2 * n * do + 2 * distinct * c["rank"] * (di + do)
            f += 2 * n * di * do + 2 * on * c["rank"] * (di + do)
        else:
            b += distinct * do * (di + 4 if i8 else 2 * di) + 2 * on * do
            f += 2 * on * di * do
    return {"bytes": b, "flops": f}


def _quantised(w):
    """int8 rows and their scales (symmetric per output channel)."""
    amax = w.abs().amax(-1, keepdim=True).clamp_min(1e-8)
    return torch.round(w * (127.0 / amax)).to(torch.int8), (amax[..., 0] / 127.0).float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std

    ids = _ids(case)
    n, fan, slots, rank = ids.size, case["fan"], case["slots"], case["rank"]
    st = {"op": case["op"], "n": n, "fan": fan, "slots": slots, "rank": rank,
          "ids": torch.from_numpy(ids).to(dev), "x": {}, "mods": []}
    # the host's view of the batch it formed: distinct slots, and each one's rows padded to the longest group
    on = np.unique(ids[ids >= 0])
    groups = [np.nonzero(ids == a)[0] for a in on]
    length = max([1] + [len(v) for v in groups])
    pad = np.full((len(on), length), n, np.int64)
    for i, v in enumerate(groups):
        pad[i, :len(v)] = v
    st["bound"] = len(on)
    st["slot_list"] = torch.from_numpy(on.astype(np.int64)).to(dev)
    st["pad"] = torch.from_numpy(pad).to(dev)
    for m, di, do in _shapes(case):
        share = _SHARE[m]
        if share not in st["x"]:
            # activations: unit normal, with a few strong channels
            gain = 1.0 + 7.0 * (torch.rand(di, generator=g, device=dev) < 1 / 256).float()
            st["x"][share] = (normal(n if fan == 1 else -(-n // fan), di) * gain).to(torch.bfloat16)
        e = {"name": m, "x": st["x"][share], "d_in": di, "d_out": do,
             "y": torch.zeros(n, do, dtype=torch.bfloat16, device=dev)}
        pitch = -(-di // 16) * 16
        if case["op"] == "linear_i8":
            e["Wq"] = torch.zeros(do, pitch, dtype=torch.int8, device=dev)
            e["Wq"][:, :di], e["Ws"] = _quantised(normal(do, di, std=di ** -0.5))
            ldb = -(-rank // 8) * 8
            e["A"] = normal(slots, rank, di, std=0.02).to(torch.bfloat16)
            e["B"] = torch.zeros(slots, do, ldb, dtype=torch.bfloat16, device=dev)
            e["B"][:, :, :rank] = normal(slots, do, rank, std=0.02).to(torch.bfloat16)
            e["scale"] = (0.5 + 1.5 * torch.rand(slots, generator=g, device=dev)).float()
        elif case["op"] == "grouped":
            e["W"] = torch.empty(slots, do, di, dtype=torch.bfloat16, device=dev)
            for a in range(slots):
                e["W"][a] = normal(do, di, std=di ** -0.5)
        else:
            e["Wq"] = torch.zeros(slots, do, pitch, dtype=torch.int8, device=dev)
            e["Ws"] = torch.empty(slots, do, dtype=torch.float32, device=dev)
            for a in range(slots):
                e["Wq"][a, :, :di], e["Ws"][a] = _quantised(normal(do, di, std=di ** -0.5))
        st["mods"].append(e)
    return st


# ---- plain form

def _rows_int8(x):
    """Each row as whole numbers of a 127th of its largest magnitude (64-bit quotients: no rounding near a tie)."""
    x = x.double()
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)))
    return q.float(), (amax / 127.0).float()


def _gathered(x, pad):
    """Rows of x for each group, [groups, d, longest], zero where a group ends (x has one zero row more)."""
    x = torch.cat([x, torch.zeros_like(x[:1])])
    return x[pad].transpose(1, 2).contiguous()


def _scattered(out, pad, yt):
    """out rows <- yt [groups, d_out, longest]; the padding goes to one row past the end."""
    ext = torch.cat([out, torch.zeros_like(out[:1])])
    ext[pad.reshape(-1)] = yt.transpose(1, 2).reshape(-1, yt.shape[1])
    return ext[:-1]


def _plain_linear(st, e):
    q, s = _rows_int8(e["x"])
    y = (q @ e["Wq"][:, :e["d_in"]].float().t()) * s * e["Ws"]
    if st["bound"]:
        xt = _gathered(e["x"].float(), st["pad"])
        v = torch.bmm(e["A"][st["slot_list"]].float(), xt)
        dl = torch.bmm(e["B"][st["slot_list"]][:, :, :st["rank"]].float().contiguous(), v)
        dl = dl * e["scale"][st["slot_list"]][:, None, None]
        y = y + _scattered(torch.zeros_like(y), st["pad"], dl)
    return y.to(torch.bfloat16)


def _plain_grouped(st, e):
    y = torch.zeros(st["n"], e["d_out"], dtype=torch.float32, device=e["x"].device)
    if not st["bound"]:
        return y.to(torch.bfloat16)
    x = e["x"].float() if st["op"] == "grouped" else None
    s = None
    if x is None:
        x, s = _rows_int8(e["x"])
    if st["fan"] > 1:
        x = x.repeat_interleave(st["fan"], 0)[:st["n"]]
        s = None if s is None else s.repeat_interleave(st["fan"], 0)[:st["n"]]
    xt = _gathered(x, st["pad"])
    if st["op"] == "grouped":
        return _scattered(y, st["pad"], torch.bmm(e["W"][st["slot_list"]].float(), xt)).to(torch.bfloat16)
    yt = torch.bmm(e["Wq"][st["slot_list"]][:, :, :e["d_in"]].float().contiguous(), xt) * e["Ws"][st["slot_list"]][:, :, None]
    return (_scattered(y, st["pad"], yt) * s).to(torch.bfloat16)


# ---- the library's calls

def _plan(st):
    """What a server keeps between steps: the device table, the projections, the segment buffers, the workspace."""
    import adapter_gemv_amd as lg
    n, slots, mods = st["n"], st["slots"], st["mods"]
    p = {"seg": lg.Segments(n, max_segments=st["bound"])}
    sum_in = sum(e["d_in"] for e in mods)
    col = {m: i for i, m in enumerate(lg.MODULES)}
    at = np.zeros((3, slots, len(lg.MODULES)), np.uint64)

    def each(t, k, e):
        at[k, :, col[e["name"]]] = t.data_ptr() + np.arange(slots, dtype=np.uint64) * np.uint64(t[0].numel() * t.element_size())

    if st["op"] == "linear_i8":
        ranks = np.zeros(at.shape[1:], np.int32)
        scales = np.ones(at.shape[1:], np.float32)
        for e in mods:
            each(e["A"], 0, e)
            each(e["B"], 1, e)
            ranks[:, col[e["name"]]] = st["rank"]
            scales[:, col[e["name"]]] = e["scale"].cpu().numpy()
        host = lg.pack_table(at[0], at[1], ranks, scales)
        p["ios"] = {e["name"]: lg.LinearI8IO(e["x"], e["Wq"], e["Ws"], e["y"]) for e in mods}
        size = lg.linear_i8_workspace_bytes(n, slots, st["rank"], sum_in, len(mods))
    else:
        ld = np.zeros(at.shape[1:], np.int64)
        for e in mods:
            each(e["W"] if st["op"] == "grouped" else e["Wq"], 0, e)
            ld[:, col[e["name"]]] = (e["W"] if st["op"] == "grouped" else e["Wq"]).shape[2]
            if st["op"] == "grouped_i8":
                each(e["Ws"], 1, e)
        host = lg.pack_weights(at[0], ld, at[1] if st["op"] == "grouped_i8" else None)
        p["ios"] = {e["name"]: lg.GroupedIO(e["x"], e["y"], rows_per_x=st["fan"]) for e in mods}
        size = lg.grouped_workspace_bytes(n, slots, sum_in, len(mods))
    p["table"] = torch.from_numpy(host.view(np.uint8).reshape(-1).copy()).to("cuda")
    p["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return p


def _own(st):
    import adapter_gemv_amd as lg
    if "plan" not in st:
        st["plan"] = _plan(st)
    p = st["plan"]
    lg.build_segments(st["ids"], st["slots"], p["seg"], p["ws"])
    if st["op"] == "linear_i8":
        lg.linear_layer(p["ios"], st["n"], st["ids"], p["table"], st["slots"], p["seg"], st["rank"], p["ws"])
    else:
        lg.grouped_layer(p["ios"], st["n"], p["table"], st["slots"], p["seg"], p["ws"], int8=st["op"] == "grouped_i8")
    return {e["name"]: e["y"] for e in st["mods"]}


def run(state):
    if own:
        return _own(state)
    f = _plain_linear if state["op"] == "linear_i8" else _plain_grouped
    return {e["name"]: f(state, e) for e in state["mods"]}


# ---- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    ids = st["ids"].long()
    out = {}
    for e in st["mods"]:
        x = e["x"].to(torch.float64)
        row = torch.arange(st["n"], device=x.device) // st["fan"]
        big = x.abs().max(dim=1).values
        if case["op"] != "grouped":
            unit = big / 127
            whole = torch.where(unit[:, None] > 0, torch.round(127 * x / big[:, None]), 0.0)
        y = torch.zeros(st["n"], e["d_out"], dtype=torch.float64, device=x.device)
        if case["op"] == "linear_i8":
            for lo in range(0, e["d_out"], 4096):
                w = e["Wq"][lo:lo + 4096, :e["d_in"]].to(torch.float64) * e["Ws"][lo:lo + 4096, None].to(torch.float64)
                y[:, lo:lo + 4096] = torch.matmul(whole, w.t()) * unit[:, None]
        for a in range(case["slots"]):
            at = torch.nonzero(ids == a)[:, 0]
            if at.numel() == 0:
                continue
            if case["op"] == "linear_i8":
                v = torch.matmul(x[at], e["A"][a].to(torch.float64).t())
                y[at] += e["scale"][a].to(torch.float64) * torch.matmul(v, e["B"][a, :, :case["rank"]].to(torch.float64).t())
            elif case["op"] == "grouped":
                y[at] = torch.matmul(x[row[at]], e["W"][a].to(torch.float64).t())
            else:
                w = e["Wq"][a, :, :e["d_in"]].to(torch.float64) * e["Ws"][a][:, None].to(torch.float64)
                y[at] = torch.matmul(whole[row[at]], w.t()) * unit[row[at]][:, None]
        out[e["name"]] = y
    return out
