"""The cases of the library's grouped FP8 products and of its 8-bit integer linear.

Three operators:

  grouped_forward   Y[r] = bf16(X8[r] W8[e]^T / (sx sw[e])) for the rows r of group e: the experts' linear of a
                    mixture of experts, rows sorted by expert, group sizes ragged and known on the device only
  grouped_backward  both of its gradients, dX[r] = G8[r] W8[e] / (sg sw[e]) and dW[e] = G8_e^T X8_e / (sg sx)
  int8_linear       Y = (q(x) W8^T) * sx[token] * sw[channel] + bias: a linear served in 8-bit integers, its input
                    quantized row by row within the call
"""
import math

import numpy as np
import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


# ---------------------------------------------------------------------------------------------- cases

def _grouped(op, groups, rows, n, k, skew):
    return {"op": op, "groups": groups, "rows": rows, "n": n, "k": k, "skew": skew}


def listed():
    fwd, bwd = "grouped_forward", "grouped_backward"
    cases = [
        # one decoding step of four tokens, one expert each: latency, and the weights of at most four experts
        ("forward_decode_4_rows", _grouped(fwd, 8, 4, 4096, 1024, 0.0)),
        # a decoding batch over many experts: two rows an expert on average, some experts idle; weight reads bound it
        ("forward_decode_128_rows_64_groups", _grouped(fwd, 64, 128, 6912, 1536, 0.5)),
        # odd sizes throughout: the last k-block, row tile and column tile are ragged, rows of Y are not 16-byte aligned
        ("forward_odd_1111_rows", _grouped(fwd, 7, 1111, 1511, 1000, 1.0)),
        # a training step's forward over the 4096 x 11008 weights, moderately unbalanced experts
        ("forward_train_8192_rows", _grouped(fwd, 8, 8192, 11008, 4096, 0.3)),
        # the backward of a short micro-batch: dW's output is most of the traffic
        ("backward_512_rows", _grouped(bwd, 8, 512, 4096, 1024, 0.3)),
        # the backward over 16 smaller experts
        ("backward_4096_rows_16_groups", _grouped(bwd, 16, 4096, 6912, 1536, 0.5)),
        # odd sizes: group ends inside dW's k-blocks
        ("backward_odd_1111_rows", _grouped(bwd, 7, 1111, 1511, 1000, 1.0)),
        # the backward of the training step above
        ("backward_train_8192_rows", _grouped(bwd, 8, 8192, 11008, 4096, 0.3)),
        # one token through a square projection: latency and one read of the weights
        ("int8_1_row", {"op": "int8_linear", "rows": 1, "n": 4096, "k": 4096, "bias": False, "dtype": "bf16"}),
        # a decoding batch through an up projection
        ("int8_16_rows", {"op": "int8_linear", "rows": 16, "n": 11008, "k": 4096, "bias": True, "dtype": "bf16"}),
        # odd sizes, half-precision activations
        ("int8_odd_333_rows", {"op": "int8_linear", "rows": 333, "n": 1511, "k": 1000, "bias": True, "dtype": "fp16"}),
        # a prompt of 8192 tokens: compute bound
        ("int8_8192_rows", {"op": "int8_linear", "rows": 8192, "n": 11008, "k": 4096, "bias": False, "dtype": "bf16"}),
    ]
    return [dict(c, name=name) for name, c in cases]


_MOST_FLOPS = 2 * 8192 * 11008 * 4096
_MOST_WEIGHTS = 8 * 11008 * 4096


def _log_int(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    """Group counts 1..64, rows 1..8192, sides 64..11008, the product of them at most the largest listed case's."""
    op = rng.choice(("grouped_forward", "grouped_backward", "int8_linear"))
    while True:
        rows, n, k = _log_int(rng, 1, 8192), _log_int(rng, 64, 11008), _log_int(rng, 64, 11008)
        if rng.random() < 0.5:  # half of the draws have sides that are whole 64s, as most models' are
            n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
        groups = 1 if op == "int8_linear" else _log_int(rng, 1, 64)
        if 2 * rows * n * k <= _MOST_FLOPS and groups * n * k <= _MOST_WEIGHTS:
            break
    if op == "int8_linear":
        return {"op": op, "rows": rows, "n": n, "k": k, "bias": rng.random() < 0.5, "dtype": rng.choice(("bf16", "fp16", "fp32"))}
    return _grouped(op, groups, rows, n, k, rng.choice((0.0, 0.3, 0.5, 1.0)))


# ---------------------------------------------------------------------------------------------- inputs

def _shares(case):
    """The experts' shares of the rows: equal for skew 0, else falling as (rank + 1)^-skew in a scattered order."""
    groups = case["groups"]
    rank = (np.arange(groups) * 5 + 3) % groups if groups % 5 else np.arange(groups)
    share = (rank + 1.0) ** -case["skew"]
    return share / share.sum()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(gen, rows, cols, std, dtype):
    """A [rows, cols] fp8 matrix whose row stride is a multiple of 16 bytes, and the scale it was quantized with."""
    x = torch.randn((rows, cols), generator=gen, device="cuda") * std
    scale = (448.0 if dtype == E4M3 else 57344.0) / x.abs().amax().clamp_min(1e-30)
    buf = torch.zeros((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
    buf[:, :cols] = (x * scale).to(dtype).view(torch.uint8)
    return buf[:, :cols], scale.reshape(1)


def prepare(case, seed):
    gen = _gen(seed)
    rows, n, k = case["rows"], case["n"], case["k"]
    if case["op"] == "int8_linear":
        dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]
        # activations with a few strong channels and tokens of different size, as layers' inputs have them
        x = torch.randn((rows, k), generator=gen, device="cuda") * torch.exp(torch.randn((rows, 1), generator=gen, device="cuda") * 0.5)
        x[:, :: max(1, k // 7)] *= 8.0
        w = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
        sw = w.abs().amax(1) / 127.0
        buf = torch.zeros((n, (k + 15) // 16 * 16), dtype=torch.int8, device="cuda")
        buf[:, :k] = torch.round(w / sw[:, None]).clamp(-127, 127).to(torch.int8)
        bias = (torch.randn(n, generator=gen, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
        return {"op": case["op"], "x": x.to(dtype), "w8": buf[:, :k], "sw": sw, "bias": bias}
    groups = case["groups"]
    counts = np.random.RandomState(seed % (1 << 31)).multinomial(rows, _shares(case))
    offsets = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    x8, sx = _codes(gen, rows, k, 1.0, E4M3)
    ld = (k + 15) // 16 * 16
    w = torch.zeros((groups, n, ld), dtype=torch.uint8, device="cuda")
    sw = torch.empty(groups, device="cuda")
    for e in range(groups):
        one, s = _codes(gen, n, k, (0.5 + e / groups) / math.sqrt(k), E4M3)
        w[e, :, :k] = one
        sw[e : e + 1] = s
    state = {"op": case["op"], "x8": x8, "sx": sx, "w8": w[:, :, :k], "sw": sw, "offsets": offsets}
    if case["op"] == "grouped_backward":
        state["g8"], state["sg"] = _codes(gen, rows, n, 1e-3, E5M2)
    return state


# ---------------------------------------------------------------------------------------------- plain forms

def _value(codes, dtype=E4M3):
    return codes.contiguous().view(dtype).float()


def _padded(rows, offsets):
    """[groups, the largest group, columns]: each group's rows, then zeros; and the (group, place) of every row."""
    at = torch.arange(rows.shape[0], device=rows.device)
    group = (at[:, None] >= offsets[None, 1:]).sum(1)
    place = at - offsets[:-1].long()[group]
    out = rows.new_zeros((offsets.numel() - 1, int((offsets[1:] - offsets[:-1]).max()), rows.shape[1]))
    out[group, place] = rows
    return out, group, place


def _plain_forward(s):
    x, group, place = _padded(_value(s["x8"]), s["offsets"])
    y = torch.bmm(x, _value(s["w8"]).transpose(1, 2))[group, place]
    return (y / (s["sx"] * s["sw"][group, None])).to(torch.bfloat16)


def _plain_backward(s):
    x, group, place = _padded(_value(s["x8"]), s["offsets"])
    g, _, _ = _padded(_value(s["g8"], E5M2), s["offsets"])
    dx = torch.bmm(g, _value(s["w8"]))[group, place] / (s["sg"] * s["sw"][group, None])
    dw = torch.bmm(g.transpose(1, 2), x) / (s["sg"] * s["sx"])
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


def _plain_int8(s):
    x = s["x"].float()
    amax = x.abs().amax(1)
    live = amax > 0
    # the codes in 64 bits: 32 would turn values that lie next to the border of two codes
    q = torch.round(x.double() * 127.0 / torch.where(live, amax, torch.ones_like(amax)).double()[:, None]).float()
    sx = torch.where(live, amax / 127.0, torch.ones_like(amax))
    y = (q @ s["w8"].float().t()) * sx[:, None] * s["sw"]
    y = y if s["bias"] is None else y + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "sx": sx}


def run(state):
    if own:
        import fp8_delayed_scaling_03_b200 as F
        if state["op"] == "grouped_forward":
            return F.grouped_mm(state["x8"], state["w8"], state["offsets"], state["sx"], state["sw"])
        if state["op"] == "grouped_backward":
            fwd = F.ForwardResult(None, state["x8"], state["w8"], state["sx"], state["sw"], None, None)
            b = F.grouped_linear_backward(state["g8"], fwd, state["offsets"], None, g_scale_in=state["sg"])
            return {"dx": b.dx, "dw": b.dw}
        r = F.linear_int8(state["x"], state["w8"], state["sw"], bias=state["bias"])
        return {"y": r.y, "sx": r.sx}
    return {"grouped_forward": _plain_forward, "grouped_backward": _plain_backward, "int8_linear": _plain_int8}[state["op"]](state)


# ---------------------------------------------------------------------------------------------- work, exact values

def work(case):
    rows, n, k = case["rows"], case["n"], case["k"]
    flops = 2.0 * rows * n * k
    if case["op"] == "int8_linear":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": size * rows * k + n * k + 4 * n + (2 * n if case["bias"] else 0) + size * rows * n + 4 * rows, "flops": flops}
    active = float((1.0 - (1.0 - _shares(case)) ** rows).sum())  # experts that get a row, on average
    weights = active * n * k
    small = 4 * (2 * case["groups"] + 2)
    if case["op"] == "grouped_forward":
        return {"bytes": rows * k + weights + 2 * rows * n + small, "flops": flops}
    return {"bytes": rows * (n + k) + weights + 2 * rows * k + 2 * case["groups"] * n * k + small, "flops": 2 * flops}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int8_linear":
        x, w, sw = s["x"].double(), s["w8"].double(), s["sw"].double()
        top = torch.amax(torch.abs(x), dim=1, keepdim=True)
        top = torch.where(top == 0, torch.full_like(top, 127.0), top)  # a row of zeros: scale 1, codes 0
        sx = top / 127.0
        y = torch.einsum("ik,jk->ij", torch.round(x * 127.0 / top), w) * (sx * sw[None, :])
        if s["bias"] is not None:
            y = y + s["bias"].double()
        return {"y": y, "sx": sx[:, 0]}
    off = s["offsets"].tolist()
    sx = s["sx"].double()
    backward = case["op"] == "grouped_backward"
    first, second = [], []
    for e in range(case["groups"]):
        x = s["x8"][off[e] : off[e + 1]].contiguous().view(E4M3).double()
        w = s["w8"][e].contiguous().view(E4M3).double()
        sw = s["sw"][e].double()
        if not backward:
            first.append(torch.einsum("rk,nk->rn", x, w) / (sx * sw))
            continue
        g = s["g8"][off[e] : off[e + 1]].contiguous().view(E5M2).double()
        first.append(torch.einsum("rn,nk->rk", g, w) / (s["sg"].double() * sw))
        second.append((torch.einsum("rn,rk->nk", g, x) / (s["sg"].double() * sx)).float())
    if not backward:
        return torch.cat(first)
    return {"dx": torch.cat(first), "dw": torch.stack(second)}
