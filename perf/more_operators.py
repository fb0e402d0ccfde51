"""Cases for training the experts' gated feed-forward and for serving it in 8-bit integers.

Each case names one operator and its sizes.  `run` makes one pass: with `own`
false in elementary torch operations in 32 bits, with `own` true through the
package's entry points, on the same state.

Rows of the experts' products lie in expert order: expert e's rows are
off_pad[e] .. off_pad[e] + counts[e] of a buffer of max_rows rows, every expert
starting on a multiple of 128; the rows between are padding, which no operator
writes.  An 8-bit matrix [rows, cols] is an int8 tensor of codes q and one
float32 scale per row, amax / 127; it stands for q * scale, with
q = 127 x / amax rounded to the nearest integer, ties to the even one.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    layer = {"H": 4096, "I": 1536, "E": 64, "k": 8}
    tiny = {"T": 128, "H": 256, "I": 512, "E": 8, "k": 2, "skew": 0.0}
    return [
        # training forward of a tiny layer, where latency counts
        {"name": "ffn_forward_tiny", "op": "ffn_forward", **tiny},
        # training forward under a skewed router: a few experts take most rows, some take none
        {"name": "ffn_forward_skewed", "op": "ffn_forward", "T": 8192, **layer, "skew": 3.0},
        # backward of the tiny layer
        {"name": "ffn_backward_tiny", "op": "ffn_backward", **tiny},
        # backward of a dense block (one expert that every token takes) with an odd number of tokens
        {"name": "ffn_backward_dense", "op": "ffn_backward", "T": 5003, "H": 2176, "I": 5760, "E": 1, "k": 1,
         "skew": 0.0},
        # backward of the 64-expert layer, about 256 rows per expert
        {"name": "ffn_backward_chunk", "op": "ffn_backward", "T": 2048, **layer, "skew": 0.0},
        # gradient of the weighted sum over a token's experts, and of the routing weights, odd sizes
        {"name": "combine_backward_odd", "op": "combine_backward", "T": 1003, "H": 1408, "E": 37, "k": 3},
        # the same for a long batch
        {"name": "combine_backward_large", "op": "combine_backward", "T": 16384, "H": 4096, "E": 128, "k": 8},
        # one decode step's tokens, quantised and read back
        {"name": "quantize_int8_decode", "op": "quantize", "rows": 64, "cols": 4096},
        # one projection of the 64-expert layer, quantised once when a checkpoint is loaded
        {"name": "weights_int8_full", "op": "weights", "E": 64, "K": 4096, "N": 1536},
        # gate/up product of a single token: the weights of its experts, one row each
        {"name": "up_int8_token", "op": "up", "T": 1, **layer, "skew": 0.0},
        # gate/up product of a long prefill, about 1024 rows per expert
        {"name": "up_int8_prefill", "op": "up", "T": 16384, "H": 4096, "I": 1536, "E": 128, "k": 8, "skew": 0.0},
        # down product of a chunk of prompts, about 256 rows per expert
        {"name": "down_int8_chunk", "op": "down", "T": 2048, **layer, "skew": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_forward", "ffn_backward", "ffn_backward", "combine_backward", "quantize", "weights", "up",
                     "down"])
    odd128 = lambda most: 128 * (2 * rng.randint(0, most) + 1)  # noqa: E731
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": odd128(15)}
    if op == "weights":
        return {"op": op, "E": rng.randint(1, 64), "K": odd128(15), "N": odd128(5)}
    E = _log_int(rng, 1, 64)
    k = rng.randint(1, min(E, 8))
    T, H = _log_int(rng, 1, 8192), odd128(15)
    if op == "combine_backward":
        return {"op": op, "T": T, "H": H, "E": E, "k": k}
    I, skew = odd128(5), rng.choice([0.0, 0.0, 1.0, 3.0])
    # no more rows (every expert padded to the longest) than the chunk of the 64-expert layer has
    T = min(T, (1 << 15) // (E if skew else 2 * k))
    return {"op": op, "T": T, "H": H, "I": I, "E": E, "k": k, "skew": skew}


# ------------------------------------------------------------------ 8-bit integers in 32 bits
def _quantize(x):
    """x [..., K] -> (codes [..., K] float32, scales [...] float32)."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    q = torch.round(x * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)))
    return q, (amax / 127.0).squeeze(-1)


# ------------------------------------------------------------------ routing of a case
def _route(case, gen, device):
    """Picks and weights [T, k], and each pick's padded row, counts, padded offsets."""
    T, E, k = case["T"], case["E"], case["k"]
    bias = case.get("skew", 0.0) * -torch.log(torch.arange(1, E + 1, dtype=torch.float32, device=device))
    logits = torch.randn((T, E), generator=gen, device=device) + bias
    top = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, picked = top.indices[:, :k].contiguous(), top.values[:, :k]
    weights = torch.exp(picked - picked[:, :1])
    weights = weights / weights.sum(-1, keepdim=True)
    flat = ids.flatten()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + 127) // 128 * 128
    off_pad = torch.cat((torch.zeros(1, dtype=torch.long, device=device), padded.cumsum(0)))
    first = counts.cumsum(0) - counts
    e = flat[order]
    row = torch.empty(T * k, dtype=torch.long, device=device)
    row[order] = off_pad[e] + torch.arange(T * k, device=device) - first[e]
    return ids, weights.contiguous(), row.reshape(T, k), counts, off_pad


def _max_rows(case):
    rows = case["T"] * case["k"]
    return 128 * ((rows + 127 * min(case["E"], rows)) // 128)


# ------------------------------------------------------------------ state
def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE)

    def zeros(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=DEVICE)

    def weights(E, K, N):
        """N(0, 1 / K), the reduction axis in the middle."""
        w = torch.empty((E, K, N), dtype=torch.bfloat16, device=DEVICE)
        for e in range(0, E, 32):
            w[e:e + 32] = normal(min(32, E - e), K, N) / math.sqrt(K)
        return w

    def codes(E, N, K):
        """Such weights in 8 bits, the reduction axis last."""
        q = zeros(E * N, K, dtype=torch.int8)
        s = zeros(E * N, dtype=torch.float32)
        for e in range(0, E, 32):
            m = min(32, E - e) * N
            a, b = _quantize((normal(m, K) / math.sqrt(K)).bfloat16())
            q[e * N:e * N + m] = a.to(torch.int8)
            s[e * N:e * N + m] = b
        return q, s

    if op == "quantize":
        R, C = case["rows"], case["cols"]
        return {"case": case, "x": normal(R, C).bfloat16(), "codes": zeros(R, C, dtype=torch.int8),
                "scales": zeros(R, dtype=torch.float32), "values": zeros(R, C)}
    if op == "weights":
        E, K, N = case["E"], case["K"], case["N"]
        return {"case": case, "w": weights(E, K, N), "codes": zeros(E * N, K, dtype=torch.int8),
                "scales": zeros(E * N, dtype=torch.float32), "values": zeros(E, N, K)}

    ids, topk_w, scatter, counts, off_pad = _route(case, gen, DEVICE)
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    R, n, row = _max_rows(case), case["T"] * case["k"], scatter.flatten()

    def rows_of(values):
        """values [T * k, cols], in slot order, at their padded rows."""
        out = zeros(R, values.shape[1], dtype=values.dtype)
        out[row] = values
        return out

    st = {"case": case, "row": row, "cap": int(counts.max()), "counts": counts.to(torch.int32),
          "off_pad": off_pad.to(torch.int32), "ws": zeros(256, dtype=torch.uint8)}
    if op == "combine_backward":
        st |= {"ids": ids.to(torch.int32), "weights": topk_w, "scatter": scatter.to(torch.int32),
               "y": rows_of(normal(n, H).bfloat16()), "dout": normal(T, H).bfloat16(), "dy": zeros(R, H),
               "dlogits": zeros(T, E, dtype=torch.float32)}
        return st
    I = case["I"]
    if op in ("up", "down"):
        K, N = (H, I) if op == "up" else (I, H)
        if op == "up":
            q, s = _quantize(normal(T, K).bfloat16())
            q, s = q.repeat_interleave(k, 0), s.repeat_interleave(k)
        else:  # what the gate/up product leaves: silu(g) * u of unit normal g and u
            q, s = _quantize((torch.nn.functional.silu(normal(n, K)) * normal(n, K)).bfloat16())
        st |= {"codes": rows_of(q.to(torch.int8)), "scales": rows_of(s.unsqueeze(-1)).squeeze(-1), "out": zeros(R, N)}
        st["w0"], st["s0"] = codes(E, N, K)
        if op == "up":
            st["w1"], st["s1"] = codes(E, N, K)
        return st
    x = rows_of(normal(T, H).bfloat16().repeat_interleave(k, 0))
    st |= {"x": x, "wg": weights(E, H, I), "wu": weights(E, H, I), "wd": weights(E, I, H)}
    if op == "ffn_forward":
        st |= {"g": zeros(R, I), "u": zeros(R, I), "h": zeros(R, I), "y": zeros(R, H)}
        # the down product takes a workspace of the layer's own size
        st["ws"] = zeros(_layer_workspace(case), dtype=torch.uint8)
        return st
    g, u = normal(n, I).bfloat16(), normal(n, I).bfloat16()
    st |= {"g": rows_of(g), "u": rows_of(u),
           "h": rows_of((torch.nn.functional.silu(g.float()) * u.float()).bfloat16()),
           # a token's gradient times its routing weight
           "dy": rows_of((normal(T, H).repeat_interleave(k, 0) * topk_w.reshape(-1, 1)).bfloat16()),
           "dg": zeros(R, I), "du": zeros(R, I), "dx": zeros(R, H),
           "dwg": zeros(E, H, I), "dwu": zeros(E, H, I), "dwd": zeros(E, I, H)}
    return st


def _layer_workspace(case):
    """At least the bytes of the layer's workspace: its row buffers and a margin for tables and alignment."""
    R, T, E, k = _max_rows(case), case["T"], case["E"], case["k"]
    return 2 * R * (2 * case["H"] + case["I"]) + 16 * R + 24 * T * k + E * (T // 8 + 64) + (1 << 16)


# ------------------------------------------------------------------ one pass
def _run_own(state):
    import combine_moe_route_04_gb300 as moe

    c = state["case"]
    op = c["op"]
    if op == "quantize":
        moe.moe_quantize_int8(state["x"], c["rows"], c["cols"], state["codes"], state["scales"])
        moe.moe_dequantize_int8(state["codes"], state["scales"], c["rows"], c["cols"], state["values"])
        return {"scales": state["scales"], "values": state["values"]}
    if op == "weights":
        moe.moe_quantize_weights_int8(state["w"], c["E"], c["K"], c["N"], state["codes"], state["scales"])
        moe.moe_dequantize_int8(state["codes"], state["scales"], c["E"] * c["N"], c["K"], state["values"])
        return {"scales": state["scales"], "values": state["values"]}
    shape = (c["T"], c["H"], c.get("I", 128), c["E"], c["k"])
    counts, off, ws = state["counts"], state["off_pad"], state["ws"]
    if op == "combine_backward":
        moe.moe_combine_backward(shape, state["y"], state["scatter"], state["ids"], state["weights"], state["dout"],
                                 state["dy"], state["dlogits"], ws)
        return {"dy": state["dy"], "dlogits": state["dlogits"]}
    if op == "up":
        moe.moe_grouped_gemm_up_int8(shape, state["codes"], state["scales"], counts, off, state["w0"], state["s0"],
                                     state["w1"], state["s1"], state["out"], ws)
        return state["out"]
    if op == "down":
        moe.moe_grouped_gemm_down_int8(shape, state["codes"], state["scales"], counts, off, state["w0"], state["s0"],
                                       state["out"], ws)
        return state["out"]
    if op == "ffn_forward":
        moe.moe_grouped_gemm_up_train(shape, state["x"], counts, off, state["wg"], state["wu"], state["g"],
                                      state["u"], state["h"], ws)
        moe.moe_grouped_gemm_down(shape, state["h"], counts, off, state["wd"], state["y"], ws)
        return {name: state[name] for name in ("g", "u", "h", "y")}
    moe.moe_grouped_gemm_down_backward(shape, state["dy"], counts, off, state["wd"], state["g"], state["u"],
                                       state["dg"], state["du"], ws)
    moe.moe_grouped_gemm_up_backward(shape, state["dg"], state["du"], counts, off, state["wg"], state["wu"],
                                     state["dx"], ws)
    moe.moe_grouped_gemm_weight_backward(shape, state["x"], state["h"], state["dg"], state["du"], state["dy"],
                                         counts, off, state["dwg"], state["dwu"], state["dwd"], ws)
    return {name: state[name] for name in ("dg", "du", "dx", "dwg", "dwu", "dwd")}


def _experts(state):
    """Index [E, cap] of every expert's rows (the longest expert has cap) and which of them are there."""
    off = state["off_pad"].long()
    at = torch.arange(state["cap"], device=off.device)
    there = at < state["counts"].unsqueeze(-1)
    return torch.where(there, off[:-1, None] + at, 0), there


def _take(x, index, there):
    return x[index].float() * there.unsqueeze(-1)


def _put(like, index, there, values):
    out = torch.zeros_like(like)
    out[index[there]] = values[there].to(like.dtype)
    return out


def _plain_combine(state):
    rows, w, ids = state["scatter"].long(), state["weights"], state["ids"].long()
    dout = state["dout"].float()
    dw = (state["y"][rows].float() * dout.unsqueeze(1)).sum(-1)
    dy = torch.zeros_like(state["y"])
    dy[rows] = (w.unsqueeze(-1) * dout.unsqueeze(1)).bfloat16()
    dlogits = torch.zeros_like(state["dlogits"])
    dlogits.scatter_(1, ids, w * (dw - (w * dw).sum(-1, keepdim=True)))
    return {"dy": dy, "dlogits": dlogits}


def _plain_product(state):
    c = state["case"]
    E = c["E"]
    index, there = _experts(state)
    x = _take(state["codes"], index, there)
    sx = state["scales"][index].unsqueeze(-1)

    def product(w, s):
        y = torch.bmm(x, w.float().unflatten(0, (E, -1)).transpose(1, 2))
        return y * sx * s.unflatten(0, (E, -1)).unsqueeze(1)

    y = product(state["w0"], state["s0"])
    if c["op"] == "up":
        y = y / (1.0 + torch.exp(-y)) * product(state["w1"], state["s1"])
    return _put(state["out"], index, there, y)


def _plain_forward(state):
    index, there = _experts(state)
    x = _take(state["x"], index, there)
    g, u = torch.bmm(x, state["wg"].float()), torch.bmm(x, state["wu"].float())
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.bmm(h, state["wd"].float())
    return {name: _put(state[name], index, there, v) for name, v in (("g", g), ("u", u), ("h", h), ("y", y))}


def _plain_backward(state):
    index, there = _experts(state)
    x, h, dy, g, u = (_take(state[name], index, there) for name in ("x", "h", "dy", "g", "u"))
    wg, wu, wd = state["wg"].float(), state["wu"].float(), state["wd"].float()
    dh = torch.bmm(dy, wd.transpose(1, 2))
    s = 1.0 / (1.0 + torch.exp(-g))
    dg, du = dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s
    dx = torch.bmm(dg, wg.transpose(1, 2)) + torch.bmm(du, wu.transpose(1, 2))
    out = {name: _put(state[name], index, there, v) for name, v in (("dg", dg), ("du", du), ("dx", dx))}
    xt = x.transpose(1, 2)
    return out | {"dwg": torch.bmm(xt, dg).bfloat16(), "dwu": torch.bmm(xt, du).bfloat16(),
                  "dwd": torch.bmm(h.transpose(1, 2), dy).bfloat16()}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("quantize", "weights"):
        q, s = _quantize(state["x"] if op == "quantize" else state["w"].transpose(1, 2))
        return {"scales": s.flatten(), "values": (q * s.unsqueeze(-1)).bfloat16()}
    if op == "combine_backward":
        return _plain_combine(state)
    if op in ("up", "down"):
        return _plain_product(state)
    return _plain_forward(state) if op == "ffn_forward" else _plain_backward(state)


# ------------------------------------------------------------------ work of one pass
def work(case):
    op = case["op"]
    if op == "quantize":  # bf16 in, the values it stands for and the scales out
        n = case["rows"] * case["cols"]
        return {"bytes": n * 4 + case["rows"] * 4, "flops": 0}
    if op == "weights":
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": n * 4 + case["E"] * case["N"] * 4, "flops": 0}
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    rows = T * k
    if op == "combine_backward":  # y and dout in, dy and dlogits out
        return {"bytes": 4 * rows * H + 2 * T * H + 4 * T * E + 12 * rows, "flops": 3 * rows * H}
    I = case["I"]
    gen = torch.Generator()
    gen.manual_seed(0)
    touched = int((_route(case, gen, "cpu")[3] > 0).sum())
    if op == "up":
        return {"bytes": 2 * touched * I * (H + 4) + rows * (H + 4) + 2 * rows * I, "flops": 4 * rows * H * I}
    if op == "down":
        return {"bytes": touched * H * (I + 4) + rows * (I + 4) + 2 * rows * H, "flops": 2 * rows * H * I}
    if op == "ffn_forward":  # x and the weights in; g, u, h and y out
        return {"bytes": 2 * rows * (2 * H + 3 * I) + 6 * touched * H * I, "flops": 6 * rows * H * I}
    # x, h, g, u, dy and the weights in; dg, du, dx and every weight's gradient out
    return {"bytes": 2 * rows * (3 * H + 5 * I) + 6 * (touched + E) * H * I, "flops": 12 * rows * H * I}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_quantize(x):
    """The nearest multiple of amax / 127 (the even one of two) in float64, and the scales."""
    b = x.double()
    amax = b.abs().amax(-1, keepdim=True)
    unit = torch.where(amax > 0, amax, torch.ones_like(amax))
    # 127 x and amax are whole multiples of a common power of two: compared without rounding
    floor = torch.floor(127.0 * b / unit)
    twice = 2.0 * (127.0 * b - floor * unit)
    up = (twice > unit) | ((twice == unit) & (floor.remainder(2.0) == 1.0))
    return {"scales": (amax / 127.0).flatten(), "values": (floor + up.double()) * (amax / 127.0)}


def _sigmoid(x):
    return torch.where(x >= 0, 1.0 / (1.0 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1.0 + torch.exp(-x.abs())))


def exact(case, seed):
    st = prepare(case, seed)
    op, E = case["op"], case.get("E", 0)
    if op == "quantize":
        return _exact_quantize(st["x"])
    if op == "weights":
        each = [_exact_quantize(st["w"][e].t()) for e in range(E)]
        return {"scales": torch.cat([v["scales"] for v in each]), "values": torch.stack([v["values"] for v in each])}
    f64 = dict(dtype=torch.float64, device=DEVICE)
    counts, off = st["counts"].tolist(), st["off_pad"].tolist()
    spans = [(e, slice(off[e], off[e] + c)) for e, c in enumerate(counts)]
    if op == "combine_backward":
        dy, dl = torch.zeros(st["y"].shape, **f64), torch.zeros((case["T"], E), **f64)
        dout, w = st["dout"].double(), st["weights"].double()
        dw = torch.empty_like(w)
        for j in range(case["k"]):
            r = st["scatter"][:, j].long()
            dw[:, j] = torch.einsum("th,th->t", st["y"][r].double(), dout)
            dy[r] = dout * w[:, j:j + 1]
        mean = torch.einsum("tk,tk->t", w, dw)
        for j in range(case["k"]):
            dl[torch.arange(case["T"], device=DEVICE), st["ids"][:, j].long()] = w[:, j] * (dw[:, j] - mean)
        return {"dy": dy, "dlogits": dl}
    if op in ("up", "down"):
        out = torch.zeros(st["out"].shape, **f64)
        N = out.shape[1]
        for e, at in spans:
            x = st["codes"][at].double() * st["scales"][at].double().unsqueeze(-1)
            y = x @ (st["w0"][e * N:e * N + N].double() * st["s0"][e * N:e * N + N].double().unsqueeze(-1)).t()
            if op == "up":
                w1 = st["w1"][e * N:e * N + N].double() * st["s1"][e * N:e * N + N].double().unsqueeze(-1)
                y = y * _sigmoid(y) * (x @ w1.t())
            out[at] = y
        return out
    names = ("g", "u", "h", "y") if op == "ffn_forward" else ("dg", "du", "dx", "dwg", "dwu", "dwd")
    out = {name: torch.zeros(st[name].shape, **f64) for name in names}
    for e, at in spans:
        x, wg, wu, wd = st["x"][at].double(), st["wg"][e].double(), st["wu"][e].double(), st["wd"][e].double()
        if op == "ffn_forward":
            g, u = x @ wg, x @ wu
            h = g * _sigmoid(g) * u
            for name, v in (("g", g), ("u", u), ("h", h), ("y", h @ wd)):
                out[name][at] = v
            continue
        g, u, dy = st["g"][at].double(), st["u"][at].double(), st["dy"][at].double()
        s = _sigmoid(g)
        dh = dy @ wd.t()
        dg, du = dh * u * (s + g * s * (1.0 - s)), dh * g * s
        out["dg"][at], out["du"][at], out["dx"][at] = dg, du, dg @ wg.t() + du @ wu.t()
        out["dwg"][e], out["dwu"][e], out["dwd"][e] = x.t() @ dg, x.t() @ du, st["h"][at].double().t() @ dy
    return out
