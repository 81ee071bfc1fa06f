"""Measured operators: the gated half of a feed-forward block (gate and up
projections, activation and product) and products with 4-bit weights and group
scales, each with one base weight and the rows' adapters, and with a whole
weight per slot.

``own`` selects the form ``run`` takes: False, elementary torch operations in
32 bits, rounded once at the end; True, the calls of ``adapter_gemv_amd``.

Formulas (row b of the batch, a = its slot id):

* gated:         g = Wg x_b + scale_a Bg_a (Ag_a x_b), u likewise, h_b = bf16(act(g) * u);
                 rows with a negative id have the base terms only.
* linear_q4:     y_b = bf16(W x_b + scale_a B_a (A_a x_b)).
* grouped_gated: h_b = bf16(act(Wg_a x_{b // fan}) * (Wu_a x_{b // fan})).
* grouped_q4:    y_b = bf16(W_a x_{b // fan}).

In the grouped forms rows with a negative id are left as they are.  Weights are
bf16, or (group > 0) 4-bit: W[n][k] = s[n][k // group] * q[n][k], q from -8 to
7, two to a byte, the even k in the low half.  act is SiLU, z sigma(z), or
GELU in its tanh form.
"""
import math

import numpy as np
import torch

own = False

# Projections of a layer: (input, output) widths by name, and which share x.
_MODS = {"q": ("d", "d"), "k": ("d", "kv"), "v": ("d", "kv"), "o": ("d", "d"),
         "gate": ("d", "ffn"), "up": ("d", "ffn"), "down": ("ffn", "d")}
_SHARE = {"q": "attn", "k": "attn", "v": "attn", "o": "o", "gate": "mlp", "up": "mlp", "down": "down"}
_ADAPTED = ("gated", "linear_q4")  # a base weight and adapters; the others: a weight per slot


def _case(name, op, rows, slots, ids, mods="gate,up", d=8192, kv=1024, ffn=28672, rank=0, group=0, act="silu", base=0.0,
          fan=1, batch=1):
    c = {"op": op, "rows": rows, "slots": slots, "ids": ids, "mods": mods, "d": d, "kv": kv, "ffn": ffn, "rank": rank,
         "group": group, "act": act, "base": base, "fan": fan, "batch": batch}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decode step's MLP input in the worst mix: 128 rows, 128 different adapters of rank 16, some rows without one
        _case("gated-decode", "gated", 128, 128, "distinct", rank=16, base=0.05),
        # prefill: 8 sequences of 128 to 2048 tokens, each with its own adapter (compute bound)
        _case("gated-prefill", "gated", 0, 8, "runs", rank=16),
        # one token of one request on a 4-bit base: the weights read once
        _case("gated-q4-one-row", "gated", 1, 1, "uniform", rank=16, group=128),
        # odd widths, odd rank, short groups, a ragged batch
        _case("gated-q4-odd", "gated", 37, 19, "uniform", d=1056, ffn=2056, rank=5, group=32, act="gelu_tanh", base=0.1),
        # the smallest call: 16 rows over 4 merged adapters of 256 x 512 (launch latency)
        _case("grouped-gated-tiny", "grouped_gated", 16, 4, "uniform", d=256, ffn=512),
        # prefill through experts: 2048 tokens, two of 8 experts each, ragged groups (compute bound)
        _case("grouped-gated-prefill", "grouped_gated", 4096, 8, "uniform", d=4096, ffn=8192, fan=2, act="gelu_tanh"),
        # decode through 4-bit experts: 64 tokens, two of 8 experts each
        _case("grouped-gated-q4-decode", "grouped_gated", 128, 8, "uniform", group=128, fan=2),
        # a longer batch through 4-bit experts, odd widths
        _case("grouped-gated-q4-odd", "grouped_gated", 1001, 6, "uniform", d=2112, ffn=4104, group=64, fan=3, base=0.05),
        # decode rows spread over 32 merged adapters in 4 bits: every slot's weight read once
        _case("grouped-q4-decode", "grouped_q4", 128, 32, "uniform", mods="q", group=128),
        # the experts' way back and the attention's projections, short groups, few rows a slot
        _case("grouped-q4-odd", "grouped_q4", 77, 13, "zipf", mods="q,k,v,o,down", d=1056, kv=72, ffn=2080, group=32),
        # one token on the attention block of a 4-bit base
        _case("linear-q4-one-row", "linear_q4", 1, 1, "uniform", mods="q,k,v,o", rank=16, group=128),
        # a decode step on every projection of a 4-bit base: 16 rows, skewed over 64 resident adapters
        _case("linear-q4-layer", "linear_q4", 16, 64, "zipf", mods="q,k,v,o,gate,up,down", rank=32, group=64, base=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limit = {}
    for c in listed():
        w, key = work(c), (c["op"], c["group"] > 0)
        f, b = limit.get(key, (0, 0))
        limit[key] = (max(f, w["flops"]), max(b, w["bytes"]))
    while True:
        op = rng.choice(["gated", "grouped_gated", "grouped_q4", "linear_q4"])
        group = rng.choice([0, 32, 64, 128]) if op in ("gated", "grouped_gated") else rng.choice([32, 64, 128])
        unit = group or 8
        mods = "gate,up" if op.endswith("gated") else rng.choice(["q", "k", "q,k,v,o", "gate,up", "down", "q,o",
                                                                  "q,k,v,o,gate,up,down"])
        d = unit * _log(rng, max(1, 256 // unit), 8192 // unit)
        kv = 8 * _log(rng, 4, max(5, d // 8))
        ffn = unit * _log(rng, max(1, d // unit), max(2, min(28672, 4 * d) // unit))
        ids = rng.choice(["uniform", "zipf", "runs"])
        rows = 0 if ids == "runs" else _log(rng, 1, 2048)
        slots = _log(rng, 1, 8 if ids == "runs" else 128 if op in _ADAPTED else 32)
        c = _case("", op, rows, slots, ids, mods=mods, d=d, kv=kv, ffn=ffn, group=group,
                  rank=rng.choice([1, 5, 8, 12, 16, 32, 48, 64]) if op in _ADAPTED else 0,
                  act=rng.choice(["silu", "gelu_tanh"]), base=rng.choice([0.0, 0.0, 0.1]),
                  fan=1 if ids == "runs" or op in _ADAPTED else rng.choice([1, 1, 2, 3]), batch=rng.randrange(1 << 30))
        held = sum(i * o for _, i, o in _shapes(c)) * (1 if op in _ADAPTED else slots)
        w = work(c)
        f, b = limit[op, group > 0]
        if w["flops"] <= f and w["bytes"] <= b and held * 2 <= 8e9:
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
    adapted = c["op"] in _ADAPTED
    b = f = 0
    seen = set()
    for m, di, do in _shapes(c):
        if _SHARE[m] not in seen:
            seen.add(_SHARE[m])
            b += 2 * di * (n if adapted else -(-n // c["fan"]))
        weight = di * do // 2 + 4 * do * (di // c["group"]) if c["group"] else 2 * di * do
        rows = n if adapted else on
        b += weight * (1 if adapted else distinct) + 2 * distinct * c["rank"] * (di + do)
        f += 2 * rows * di * do + 2 * on * c["rank"] * (di + do)
        if not c["op"].endswith("gated") or m == "gate":  # the gated forms write one matrix
            b += 2 * rows * do
    return {"bytes": b, "flops": f}


def _packed(w, group):
    """4-bit rows (two values to a byte) and their group scales: symmetric, the largest magnitude at 7."""
    do, di = w.shape
    w = w.view(do, di // group, group)
    s = (w.abs().amax(-1) / 7.0).clamp_min(1e-8)
    q = torch.round(w / s[..., None]).clamp_(-8, 7).to(torch.int32).view(do, di)
    return ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8), s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std

    ids = _ids(case)
    n, fan, slots, rank, group = ids.size, case["fan"], case["slots"], case["rank"], case["group"]
    st = {"op": case["op"], "n": n, "fan": fan, "slots": slots, "rank": rank, "group": group, "act": case["act"],
          "ids": torch.from_numpy(ids).to(dev), "mods": []}
    # the host's view of the batch it formed: the distinct slots and the rows of each
    st["groups"] = [(int(a), torch.from_numpy(np.nonzero(ids == a)[0]).to(dev)) for a in np.unique(ids[ids >= 0])]
    xs = {}
    for m, di, do in _shapes(case):
        share = _SHARE[m]
        if share not in xs:
            # activations: unit normal, with a few strong channels
            gain = 1.0 + 7.0 * (torch.rand(di, generator=g, device=dev) < 1 / 256).float()
            xs[share] = (normal(n if fan == 1 else -(-n // fan), di) * gain).to(torch.bfloat16)
        e = {"name": m, "x": xs[share], "d_in": di, "d_out": do, "W": [], "s": []}
        for _ in range(1 if case["op"] in _ADAPTED else slots):
            w = normal(do, di, std=di ** -0.5)
            if group:
                q, s = _packed(w, group)
                pitch = -(-di // 32) * 16  # bytes of a row
                e["W"].append(torch.zeros(do, pitch, dtype=torch.uint8, device=dev))
                e["W"][-1][:, :di // 2] = q
                e["s"].append(s)
            else:
                e["W"].append(w.to(torch.bfloat16))
        if case["op"] in _ADAPTED:
            ldb = -(-rank // 8) * 8
            e["A"] = normal(slots, rank, di, std=0.02).to(torch.bfloat16)
            e["B"] = torch.zeros(slots, do, ldb, dtype=torch.bfloat16, device=dev)
            e["B"][:, :, :rank] = normal(slots, do, rank, std=0.02).to(torch.bfloat16)
            e["scale"] = (0.5 + 1.5 * torch.rand(slots, generator=g, device=dev)).float()
        e["y"] = torch.zeros(n, do, dtype=torch.bfloat16, device=dev)
        st["mods"].append(e)
    return st


# ---- plain form

def _weight(st, e, a, dtype=torch.float32):
    """Slot a's weight, whole."""
    w = e["W"][a]
    if not st["group"]:
        return w.to(dtype)
    w = w[:, :e["d_in"] // 2].to(torch.int32)
    q = torch.stack([w & 15, w >> 4], -1).view(w.shape[0], -1)
    q = torch.where(q > 7, q - 16, q).to(dtype)
    return (q.view(w.shape[0], -1, st["group"]) * e["s"][a].to(dtype)[..., None]).view(w.shape[0], -1)


def _plain_sums(st, e):
    """The projection's rows in 32 bits, before activation and rounding."""
    x = e["x"].float()
    if st["op"] in _ADAPTED:
        y = x @ _weight(st, e, 0).t()
        for a, at in st["groups"]:
            v = x[at] @ e["A"][a].float().t()
            y[at] += e["scale"][a] * (v @ e["B"][a, :, :st["rank"]].float().t())
        return y
    y = torch.zeros(st["n"], e["d_out"], dtype=torch.float32, device=x.device)
    for a, at in st["groups"]:
        y[at] = x[torch.div(at, st["fan"], rounding_mode="floor")] @ _weight(st, e, a).t()
    return y


def _act(z, kind):
    t = z if kind == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1.0 + torch.exp(-t))


def _plain(st):
    if not st["op"].endswith("gated"):
        return {e["name"]: _plain_sums(st, e).to(torch.bfloat16) for e in st["mods"]}
    gate, up = (_plain_sums(st, e) for e in st["mods"])
    return {"h": (_act(gate, st["act"]) * up).to(torch.bfloat16)}


# ---- the library's calls

def _plan(st):
    """What a server keeps between steps: the device table, the projections, the segment buffers, the workspace."""
    import adapter_gemv_amd as lg
    n, slots, mods, rank, group = st["n"], st["slots"], st["mods"], st["rank"], st["group"]
    p = {"seg": lg.Segments(n, max_segments=len(st["groups"]))}
    sum_in = sum(e["d_in"] for e in mods)
    col = {m: i for i, m in enumerate(lg.MODULES)}
    shape = (slots, len(lg.MODULES))
    at = np.zeros((2,) + shape, np.uint64)
    ld = np.zeros((2,) + shape, np.int64)
    if st["op"] in _ADAPTED:
        ranks, scales = np.zeros(shape, np.int32), np.ones(shape, np.float32)
        for e in mods:
            for k, t in enumerate((e["A"], e["B"])):
                at[k, :, col[e["name"]]] = t.data_ptr() + np.arange(slots, dtype=np.uint64) * np.uint64(2 * t[0].numel())
            ranks[:, col[e["name"]]] = rank
            scales[:, col[e["name"]]] = e["scale"].cpu().numpy()
        host = lg.pack_table(at[0], at[1], ranks, scales)
        if st["op"] == "linear_q4":
            p["ios"] = {e["name"]: lg.LinearQ4GIO(e["x"], e["W"][0], e["s"][0], e["y"], group) for e in mods}
            size = lg.linear_q4g_workspace_bytes(n, slots, rank, sum_in, len(mods))
        else:
            gate, up = mods
            if group:
                p["ios"] = lg.GatedQ4GIO(gate["x"], gate["W"][0], gate["s"][0], up["W"][0], up["s"][0], gate["y"], group)
            else:
                p["ios"] = lg.GatedIO(gate["x"], gate["W"][0], up["W"][0], gate["y"])
            size = lg.gated_workspace_bytes(n, slots, rank, gate["d_in"])
    else:
        for e in mods:
            for a in range(slots):
                at[0, a, col[e["name"]]] = e["W"][a].data_ptr()
                ld[0, a, col[e["name"]]] = e["W"][a].stride(0)
                if group:
                    at[1, a, col[e["name"]]] = e["s"][a].data_ptr()
                    ld[1, a, col[e["name"]]] = e["s"][a].stride(0)
        host = lg.pack_weights_q4g(at[0], ld[0], at[1], ld[1]) if group else lg.pack_weights(at[0], ld[0])
        ios = {e["name"]: lg.GroupedIO(e["x"], e["y"], rows_per_x=st["fan"]) for e in mods}
        p["ios"] = ios if st["op"] == "grouped_q4" else ios["gate"]
        size = lg.workspace_bytes(n, slots, 1, 0)
    p["table"] = torch.from_numpy(host.view(np.uint8).reshape(-1).copy()).to("cuda")
    p["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return p


def _own(st):
    import adapter_gemv_amd as lg
    if "plan" not in st:
        st["plan"] = _plan(st)
    p, n, slots = st["plan"], st["n"], st["slots"]
    lg.build_segments(st["ids"], slots, p["seg"], p["ws"])
    if st["op"] == "linear_q4":
        lg.linear_layer(p["ios"], n, st["ids"], p["table"], slots, p["seg"], st["rank"], p["ws"])
    elif st["op"] == "gated":
        lg.gated_layer(p["ios"], n, st["ids"], p["table"], slots, p["seg"], st["rank"], p["ws"], activation=st["act"])
    elif st["op"] == "grouped_q4":
        lg.grouped_layer_q4g(p["ios"], n, p["table"], slots, p["seg"], st["group"])
    elif st["group"]:
        lg.grouped_gated_layer_q4g(p["ios"], n, p["table"], slots, p["seg"], st["group"], activation=st["act"])
    else:
        lg.grouped_gated_layer(p["ios"], n, p["table"], slots, p["seg"], activation=st["act"])
    if st["op"].endswith("gated"):
        return {"h": st["mods"][0]["y"]}
    return {e["name"]: e["y"] for e in st["mods"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    ids = st["ids"].long()
    group, f64 = case["group"], torch.float64
    sums = {}
    for e in st["mods"]:
        x = e["x"].to(f64).repeat_interleave(case["fan"], 0)[:st["n"]]
        y = torch.zeros(st["n"], e["d_out"], dtype=f64, device=x.device)
        for a in ([-1] if case["op"] in _ADAPTED else []) + list(range(case["slots"])):
            at = torch.arange(st["n"], device=x.device) if a < 0 else torch.nonzero(ids == a)[:, 0]
            if at.numel() == 0:
                continue
            if a >= 0 and case["op"] in _ADAPTED:
                v = torch.matmul(x[at], e["A"][a].to(f64).t())
                y[at] += e["scale"][a].to(f64) * torch.matmul(v, e["B"][a, :, :case["rank"]].to(f64).t())
                continue
            for lo in range(0, e["d_out"], 4096):  # some outputs at a time
                w = e["W"][max(a, 0)][lo:lo + 4096]
                if group:
                    low, high = torch.remainder(w, 16).to(f64), torch.div(w, 16, rounding_mode="floor").to(f64)
                    whole = torch.zeros(w.shape[0], 2 * w.shape[1], dtype=f64, device=w.device)
                    whole[:, 0::2], whole[:, 1::2] = low - 16 * (low >= 8), high - 16 * (high >= 8)
                    w = whole[:, :e["d_in"]] * e["s"][max(a, 0)][lo:lo + 4096].to(f64).repeat_interleave(group, 1)
                y[at, lo:lo + 4096] = torch.matmul(x[at], w.to(f64).t())
        sums[e["name"]] = y
    if not case["op"].endswith("gated"):
        return sums
    z = sums["gate"]
    if case["act"] == "silu":
        a = z * torch.sigmoid(z)
    else:
        a = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return {"h": a * sums["up"]}
