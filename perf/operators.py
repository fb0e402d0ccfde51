"""Cases for the layer's MXFP4 quantisation and products and for the router's balance loss.

Each case names one operator and its sizes.  `run` makes one pass: with `own`
false in elementary torch operations in 32 bits, with `own` true through the
package's entry points, on the same state.

Formats (those of the package): an MXFP4 matrix [rows, cols] is a uint8 tensor
of codes [rows, cols / 2] (element 2i in the low nibble of byte i; e2m1: sign,
then 0 0.5 1 1.5 2 3 4 6) and one scale byte s per 32 columns, standing for
2^(s - 127), in tiles of 128 rows x 4 blocks: [rows / 128][cols / 128][32][4][4]
= (row block, column block, row % 32, row % 128 / 32, block % 4).
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's tokens of the 4096-wide layer, quantised and read back
        {"name": "quantize_decode", "op": "quantize", "rows": 64, "cols": 4096},
        # a prefill's tokens of the same layer
        {"name": "quantize_prefill", "op": "quantize", "rows": 16384, "cols": 4096},
        # a small layer's weights with sizes that are not powers of two
        {"name": "weights_ragged", "op": "weights", "E": 7, "K": 1408, "N": 640},
        # one projection of the 64-expert layer, quantised once when a checkpoint is loaded
        {"name": "weights_full", "op": "weights", "E": 64, "K": 4096, "N": 1536},
        # gate/up product of one decode step: every expert's weights for about 8 rows each
        {"name": "up_decode", "op": "up", "T": 64, "H": 4096, "I": 1536, "E": 64, "k": 8, "skew": 0.0},
        # gate/up product of a chunk of prompts, about 256 rows per expert
        {"name": "up_chunk", "op": "up", "T": 2048, "H": 4096, "I": 1536, "E": 64, "k": 8, "skew": 0.0},
        # gate/up product of a long prefill, about 1024 rows per expert
        {"name": "up_prefill", "op": "up", "T": 16384, "H": 4096, "I": 1536, "E": 128, "k": 8, "skew": 0.0},
        # down product of a tiny layer, where latency counts
        {"name": "down_tiny", "op": "down", "T": 128, "H": 256, "I": 512, "E": 8, "k": 2, "skew": 0.0},
        # down product under a skewed router: a few experts take most rows, some take none
        {"name": "down_skewed", "op": "down", "T": 8192, "H": 4096, "I": 1536, "E": 64, "k": 8, "skew": 3.0},
        # balance loss and gradient of a tiny router
        {"name": "balance_tiny", "op": "balance", "T": 128, "E": 8, "k": 2, "masked": False},
        # odd token and expert counts, padding tokens masked out
        {"name": "balance_odd", "op": "balance", "T": 5003, "E": 37, "k": 3, "masked": True},
        # a training batch of a wide router, padding tokens masked out
        {"name": "balance_large", "op": "balance", "T": 262144, "E": 256, "k": 8, "masked": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "weights", "up", "down", "balance"])
    odd128 = lambda most: 128 * (2 * rng.randint(0, most) + 1)  # noqa: E731
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": odd128(15)}
    if op == "weights":
        return {"op": op, "E": rng.randint(1, 64), "K": odd128(15), "N": odd128(5)}
    if op == "balance":
        E = rng.randint(1, 256)
        return {"op": op, "T": _log_int(rng, 1, 262144), "E": E, "k": rng.randint(1, min(E, 16)),
                "masked": rng.random() < 0.5}
    E = _log_int(rng, 1, 128)
    return {"op": op, "T": _log_int(rng, 1, 8192), "H": odd128(15), "I": odd128(5), "E": E,
            "k": rng.randint(1, min(E, 8)), "skew": rng.choice([0.0, 0.0, 1.0, 3.0])}


# ------------------------------------------------------------------ MXFP4 in 32 bits
def _e2m1_values(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        dtype=torch.float32, device=device)


def _quantize(x):
    """x [..., K] -> (values of the elements before scaling [..., K] float32, scale bytes [..., K / 32])."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    exponent = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    y = torch.ldexp(b, -exponent.unsqueeze(-1))
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(y / step) * step).clamp(-6.0, 6.0)
    return q.flatten(-2), (exponent + 127).to(torch.uint8)


def _pack(q):
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _tile(s):
    """Scale bytes [..., rows, K / 32] in the tiled layout (rows a multiple of 128)."""
    s = s.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 4, 32))
    n = s.dim()
    return s.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).contiguous()


def _untile(s):
    n = s.dim()
    return s.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).flatten(-5, -3).flatten(-2)


def _scale(s):
    return torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 127)


def _decode(codes, tiles):
    """The float32 values [..., rows, K] that codes and tiled scales stand for."""
    lut = _e2m1_values(codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    scale = _scale(_untile(tiles))
    return (v.unflatten(-1, (-1, BLOCK)) * scale.unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ routing of a case
def _top_k(logits, k):
    return torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k].to(torch.int32)


def _logits(T, E, skew, gen, device):
    bias = skew * -torch.log(torch.arange(1, E + 1, dtype=torch.float32, device=device))
    return torch.randn((T, E), generator=gen, device=device) + bias


def _route(case, gen, device):
    """(token of each routed row in expert order, its padded row, counts, padded offsets)."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = _top_k(_logits(T, E, case["skew"], gen, device), k).flatten().long()
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    padded = (counts + 127) // 128 * 128
    off_pad = torch.cat((torch.zeros(1, dtype=torch.long, device=device), padded.cumsum(0)))
    first = counts.cumsum(0) - counts
    e = ids[order]
    row = off_pad[e] + torch.arange(T * k, device=device) - first[e]
    return order // k, row, counts, off_pad


def _max_rows(case):
    rows = case["T"] * case["k"]
    return 128 * ((rows + 127 * min(case["E"], rows)) // 128)


# ------------------------------------------------------------------ state
def _weights(E, N, K, gen):
    """Random weights N(0, 1/K) in MXFP4, each expert's [N, K] with the reduction axis last."""
    codes, tiles = [], []
    for e0 in range(0, E, 32):
        w = torch.randn((min(32, E - e0), N, K), generator=gen, device=DEVICE) / math.sqrt(K)
        q, s = _quantize(w)
        codes.append(_pack(q))
        tiles.append(_tile(s))
    return torch.cat(codes), torch.cat(tiles)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    u8 = dict(dtype=torch.uint8, device=DEVICE)
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        return {"case": case, "x": torch.randn((R, C), generator=gen, device=DEVICE).bfloat16(),
                "codes": torch.zeros((R, C // 2), **u8),
                "scales": torch.zeros(((R + 127) // 128, C // 128, 32, 4, 4), **u8),
                "values": torch.zeros((R, C), dtype=torch.bfloat16, device=DEVICE)}
    if op == "weights":
        E, K, N = case["E"], case["K"], case["N"]
        w = torch.randn((E, K, N), generator=gen, device=DEVICE).mul_(1.0 / math.sqrt(K)).bfloat16()
        return {"case": case, "w": w, "codes": torch.zeros((E, N, K // 2), **u8),
                "scales": torch.zeros((E, N // 128, K // 128, 32, 4, 4), **u8),
                "values": torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEVICE)}
    if op == "balance":
        T, E = case["T"], case["E"]
        logits = _logits(T, E, 0.25, gen, DEVICE)
        mask = (torch.rand((T,), generator=gen, device=DEVICE) < 0.85) if case["masked"] else None
        f32 = dict(dtype=torch.float32, device=DEVICE)
        i32 = dict(dtype=torch.int32, device=DEVICE)
        return {"case": case, "logits": logits, "ids": _top_k(logits, case["k"]).contiguous(), "mask": mask,
                # the loss terms' weights in the training objective
                "grad": torch.tensor([1e-2, 1e-3], **f32),
                "counts": torch.zeros(E, **i32), "num_tokens": torch.zeros(1, **i32),
                "mean_probs": torch.zeros(E, **f32), "losses": torch.zeros(2, **f32),
                "dlogits": torch.zeros((T, E), **f32), "ws": torch.zeros(1 << 20, **u8)}
    # the grouped products
    T, H, I, E = case["T"], case["H"], case["I"], case["E"]
    token, row, counts, off_pad = _route(case, gen, DEVICE)
    R = _max_rows(case)
    K, N = (H, I) if op == "up" else (I, H)
    if op == "up":
        q, s = _quantize(torch.randn((T, K), generator=gen, device=DEVICE).bfloat16())
        q, s = _pack(q)[token], s[token]
    else:
        # what the gate/up product leaves: silu(g) * u of unit normal g and u
        g = torch.randn((T * case["k"], K), generator=gen, device=DEVICE)
        h = torch.nn.functional.silu(g) * torch.randn((T * case["k"], K), generator=gen, device=DEVICE)
        q, s = _quantize(h.bfloat16())
        q = _pack(q)
    codes = torch.zeros((R, K // 2), **u8)
    codes[row] = q
    flat = torch.zeros((R, K // BLOCK), **u8)
    flat[row] = s
    state = {"case": case, "codes": codes, "scales": _tile(flat), "row": row, "cap": int(counts.max()),
             "counts": counts.to(torch.int32), "off_pad": off_pad.to(torch.int32),
             "out": torch.zeros((R, N), dtype=torch.bfloat16, device=DEVICE), "ws": torch.zeros(256, **u8)}
    state["w0"], state["s0"] = _weights(E, N, K, gen)
    if op == "up":
        state["w1"], state["s1"] = _weights(E, N, K, gen)
    return state


# ------------------------------------------------------------------ one pass
def _run_own(state):
    import combine_moe_route_04_gb300 as moe

    c = state["case"]
    op = c["op"]
    if op == "quantize":
        moe.moe_quantize_mxfp4(state["x"], c["rows"], c["cols"], state["codes"], state["scales"])
        moe.moe_dequantize_mxfp4(state["codes"], state["scales"], c["rows"], c["cols"], state["values"])
        return state["values"]
    if op == "weights":
        moe.moe_quantize_weights_mxfp4(state["w"], c["E"], c["K"], c["N"], state["codes"], state["scales"])
        moe.moe_dequantize_mxfp4(state["codes"], state["scales"], c["E"] * c["N"], c["K"], state["values"])
        return state["values"]
    if op == "balance":
        shape = (c["T"], 128, 128, c["E"], c["k"])
        moe.moe_balance_loss(shape, state["logits"], state["ids"], state["mask"], state["counts"],
                             state["num_tokens"], state["mean_probs"], state["losses"], state["ws"])
        moe.moe_balance_loss_backward(shape, state["logits"], state["mask"], state["counts"], state["num_tokens"],
                                      state["grad"], state["dlogits"])
        return {k: state[k] for k in ("counts", "num_tokens", "mean_probs", "losses", "dlogits")}
    shape = (c["T"], c["H"], c["I"], c["E"], c["k"])
    if op == "up":
        moe.moe_grouped_gemm_up_mxfp4(shape, state["codes"], state["scales"], state["counts"], state["off_pad"],
                                      state["w0"], state["s0"], state["w1"], state["s1"], state["out"], state["ws"])
    else:
        moe.moe_grouped_gemm_down_mxfp4(shape, state["codes"], state["scales"], state["counts"], state["off_pad"],
                                        state["w0"], state["s0"], state["out"], state["ws"])
    return state["out"]  # padding rows are not written: they keep their zeros


def _plain_balance(state):
    c = state["case"]
    E, k = c["E"], c["k"]
    logits, ids = state["logits"], state["ids"].long()
    part = torch.ones(c["T"], dtype=torch.bool, device=logits.device) if state["mask"] is None else state["mask"]
    n = part.sum()
    counts = torch.zeros(E, dtype=torch.int32, device=logits.device)
    counts.index_add_(0, ids.flatten(), part.int().repeat_interleave(k))
    top = logits.amax(-1, keepdim=True)
    x = torch.exp(logits - top)
    total = x.sum(-1, keepdim=True)
    w = part.float().unsqueeze(-1)
    p = x / total * w
    lse = (torch.log(total) + top) * w
    inv = torch.where(n > 0, 1.0 / n.clamp(min=1).float(), torch.zeros((), device=logits.device))
    f = counts.float() * (inv / k)
    mean_probs = p.sum(0) * inv
    losses = torch.stack((E * (f * mean_probs).sum(), (lse * lse).sum() * inv))
    d = f - (p * f).sum(-1, keepdim=True)
    dlogits = p * (state["grad"][0] * E * inv * d + state["grad"][1] * 2.0 * inv * lse)
    return {"counts": counts, "num_tokens": n.to(torch.int32).reshape(1), "mean_probs": mean_probs,
            "losses": losses, "dlogits": dlogits}


def _plain_product(state):
    c = state["case"]
    E = c["E"]
    rows = _decode(state["codes"], state["scales"])
    off = state["off_pad"].long()
    at = torch.arange(state["cap"], device=off.device)
    index = (off[:-1, None] + at).clamp(max=rows.shape[0] - 1)  # rows past an expert's count are dropped below
    x = rows[index]
    if c["op"] == "up":
        g = torch.bmm(x, _decode(state["w0"], state["s0"]).transpose(1, 2))
        u = torch.bmm(x, _decode(state["w1"], state["s1"]).transpose(1, 2))
        y = g / (1.0 + torch.exp(-g)) * u
    else:
        y = torch.bmm(x, _decode(state["w0"], state["s0"]).transpose(1, 2))
    e = torch.bucketize(state["row"], off[1:], right=True).clamp(max=E - 1)
    out = torch.zeros((rows.shape[0], y.shape[-1]), dtype=torch.bfloat16, device=y.device)
    out[state["row"]] = y[e, state["row"] - off[e]].bfloat16()
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("quantize", "weights"):
        q, s = _quantize(state["x"] if op == "quantize" else state["w"].transpose(1, 2))
        scale = _scale(s)
        return (q.unflatten(-1, (-1, BLOCK)) * scale.unsqueeze(-1)).flatten(-2).bfloat16()
    if op == "balance":
        return _plain_balance(state)
    return _plain_product(state)


# ------------------------------------------------------------------ work of one pass
_PACKED = 0.5 + 1.0 / BLOCK  # bytes per MXFP4 element, its share of the scale included


def work(case):
    op = case["op"]
    if op == "quantize":  # bf16 in, the values it stands for out
        n = case["rows"] * case["cols"]
        return {"bytes": n * 4, "flops": 0}
    if op == "weights":
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": n * 4, "flops": 0}
    if op == "balance":
        n = case["T"] * case["E"]
        return {"bytes": n * 8 + 4 * case["T"] * case["k"] + (case["T"] if case["masked"] else 0) + 8 * case["E"],
                "flops": 12 * n}
    gen = torch.Generator()
    gen.manual_seed(0)
    counts = _route(case, gen, "cpu")[2]
    touched, rows = int((counts > 0).sum()), case["T"] * case["k"]
    K, N = (case["H"], case["I"]) if case["op"] == "up" else (case["I"], case["H"])
    mats = 2 if case["op"] == "up" else 1
    return {"bytes": mats * touched * N * K * _PACKED + rows * K * _PACKED + rows * N * 2,
            "flops": 2 * mats * rows * N * K}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_quantize(x):
    """The nearest element of each block's grid (ties to the even code), scale included, in float64."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, torch.exp2(torch.floor(torch.log2(amax)) - 2), torch.ones_like(amax))
    a = b.abs() / scale
    # between neighbours v_i < v_{i+1} the larger one is taken above their middle, and at it where its code is even
    out = torch.zeros_like(a)
    grid = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    for i in range(1, 8):
        middle = (grid[i - 1] + grid[i]) / 2
        out = torch.where((a >= middle) if i % 2 == 0 else (a > middle), torch.full_like(a, grid[i]), out)
    return (torch.copysign(out, b) * scale).flatten(-2)


def _exact_decode(codes, tiles):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack((lo, hi), -1).flatten(-2)
    m, ex, sign = (c & 1).double(), (c >> 1) & 3, (c >> 3).double()
    v = torch.where(ex == 0, m * 0.5, (1 + m * 0.5) * torch.exp2(ex.double() - 1)) * (1 - 2 * sign)
    n = tiles.dim()
    s = tiles.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).flatten(-5, -3).flatten(-2)
    return v * torch.exp2(s.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(st["x"])
    if op == "weights":
        return torch.stack([_exact_quantize(st["w"][e].t()) for e in range(case["E"])])
    if op == "balance":
        logits, ids, E, k = st["logits"].double(), st["ids"].long(), case["E"], case["k"]
        use = torch.ones(case["T"], dtype=torch.bool, device=logits.device) if st["mask"] is None else st["mask"]
        n = int(use.sum())
        dl = torch.zeros_like(logits)
        if n == 0:
            zero = torch.zeros(E, dtype=torch.float64, device=logits.device)
            return {"counts": zero.int(), "num_tokens": zero[:1].int(), "mean_probs": zero,
                    "losses": torch.zeros(2, dtype=torch.float64, device=logits.device), "dlogits": dl}
        p = torch.softmax(logits[use], -1)
        lse = torch.logsumexp(logits[use], -1)
        counts = torch.bincount(ids[use].flatten(), minlength=E)
        f = counts.double() / (n * k)
        g0, g1 = st["grad"].double()
        dl[use] = (g0 * E / n * p * (f - (p @ f).unsqueeze(-1)) + g1 * 2 / n * lse.unsqueeze(-1) * p)
        P = p.mean(0)
        return {"counts": counts.int(), "num_tokens": torch.tensor([n], dtype=torch.int32),
                "mean_probs": P, "losses": torch.stack((E * (f * P).sum(), (lse ** 2).mean())), "dlogits": dl}
    counts, off = st["counts"].tolist(), st["off_pad"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=st["out"].device)
    for e, c in enumerate(counts):
        if c == 0:
            continue
        b0, b1 = off[e] // 128, off[e + 1] // 128
        x = _exact_decode(st["codes"][off[e]:off[e + 1]], st["scales"][b0:b1])[:c]
        y = x @ _exact_decode(st["w0"][e], st["s0"][e]).t()
        if op == "up":
            y = torch.nn.functional.silu(y) * (x @ _exact_decode(st["w1"][e], st["s1"][e]).t())
        out[off[e]:off[e] + c] = y
    return out
